"""Which kernel the 8-bit products and input gradients take, asked on the CPU."""
import ctypes

import pytest

import int8_paths as P


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    return P.build_rule(tmp_path_factory.mktemp("rule"))


@pytest.mark.parametrize("case", P.PRODUCTS, ids=P.named)
def test_product_takes_its_path(rule, case):
    path, m, k, ns = case
    assert P.product_path(rule, m, k, ns) == path and not P.decodes(rule, m, k)


def test_decode_limit(rule):
    assert P.decodes(rule, 1, 16384) and P.decodes(rule, 4, 4096) and P.decodes(rule, 3, 5440)
    assert not P.decodes(rule, 1, 16448) and not P.decodes(rule, 4, 4160) and not P.decodes(rule, 5, 64)


@pytest.mark.parametrize("case", P.GRADIENTS + P.ADAPTED_GRADIENTS, ids=P.named)
def test_gradient_takes_its_path(rule, case):
    path, m, k, ns = case
    assert P.gradient_path(rule, m, k, ns) == path


def test_every_path_has_sizes():
    """Alone and in a set of several weights, where the rule has the path for both."""
    for count in (False, True):
        assert {c[0] for c in P.PRODUCTS if (len(c[3]) > 1) == count} >= P.PRODUCT_PATHS - (
            {"split 128x128 odd"} if count else set())
    assert {c[0] for c in P.GRADIENTS} == P.GRADIENT_PATHS
    assert {c[0] for c in P.PRODUCTS} == P.PRODUCT_PATHS


def test_a_split_needs_its_workspace(rule):
    """Without room for partial sums nothing is split, and the library asks for room
    where the rule splits."""
    import group_wise_minmax_amd as L
    for path, m, k, ns in P.PRODUCTS:
        assert not P.product_path(rule, m, k, ns, split=False).startswith("split")
        if len(ns) == 1:
            d = L.make_desc("int8", ns[0], k)
            need = L.lib.lbq_linear_fwd_tokens_workspace_bytes(ctypes.byref(d), m)
            assert (need > 0) == path.startswith("split")
    for path, m, k, ns in P.GRADIENTS:
        assert "ranges" not in P.gradient_path(rule, m, k, ns, split=False)
        descs = (L.Desc * len(ns))(*[L.make_desc("int8", n, k) for n in ns])
        need = L.lib.lbq_linear_bwd_dx_grouped_workspace_bytes(len(ns), descs, m)
        assert (need > 0) == path.endswith("ranges")
