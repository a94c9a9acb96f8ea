// The dispatch rule of the 8-bit products and input gradients, for the CPU tests.
#include "lbq_i8_choice.h"

extern "C" {

// Whether the product's own launch quantizes the tokens.
int i8_decodes(int64_t m, int64_t k) { return lbq::i8_decode_fits(m, k); }

// out: tn, tm, whole, cut, ks, per, tiles or pieces that are not whole
void i8_product_path(const int64_t* ns, int count, int64_t k, int64_t m, int split, int64_t* out) {
  const lbq::I8Choice c = lbq::i8_choose(ns, count, k, m, split != 0);
  const int64_t tiles = (int64_t)c.plan.nx * c.plan.ny;
  const int64_t rest = c.plan.whole > 0 ? (tiles - c.plan.whole) * c.plan.cut : tiles;
  const int64_t v[7] = {c.tn, c.tm, c.plan.whole, c.plan.cut, c.plan.ks, c.plan.per, rest};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}

// out: tm, ks, per, bk, bm
void i8_gradient_path(const int64_t* ns, int count, int64_t k, int64_t m, int split, int64_t* out) {
  const lbq::I8DxChoice c = lbq::i8_dx_choose(ns, count, k, m, split != 0);
  const int64_t v[5] = {c.tm, c.ks, c.per, c.bk, c.bm};
  for (int i = 0; i < 5; ++i) out[i] = v[i];
}
}
