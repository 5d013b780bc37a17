"""link_linears: a maximum has one giver and one taker.  A second taker would leave the first one's
scale to a maximum that nothing writes, a second giver would overwrite the first one's."""
import pytest


def layers(kind, count, K, N):
    import quantised_gemm_gb300 as q
    if kind == "norm":
        return [q.LayerNorm(32, K, device="cpu") for _ in range(count)]
    return [q.Fp8Linear(32, K, N, device="cpu") for _ in range(count)]


@pytest.mark.parametrize("giver,taker", [("fp8", "fp8"), ("norm", "fp8"), ("fp8", "norm")])
def test_a_second_taker_is_refused(giver, taker):
    import quantised_gemm_gb300 as q
    prev, = layers(giver, 1, 64, 64)
    first, second = layers(taker, 2, 64, 96)
    q.link_linears(prev, first)
    q.link_linears(prev, first)  # the same again
    to = (prev.y_amax_to, getattr(prev, "sdy", None) and prev.sdy.amax_algo)
    with pytest.raises(ValueError):
        q.link_linears(prev, second)
    assert prev.y_amax_to is to[0]
    assert getattr(second, "dx_amax_to") is None
    if taker == "fp8":
        assert prev.y_amax_to.data_ptr() == first.sx.amax.data_ptr()
        assert first.sx.amax_algo == q.AMAX_PRECOMPUTED and second.sx.amax_algo != q.AMAX_PRECOMPUTED


@pytest.mark.parametrize("giver,taker", [("fp8", "fp8"), ("norm", "fp8"), ("fp8", "norm")])
def test_a_second_giver_is_refused(giver, taker):
    import quantised_gemm_gb300 as q
    first, second = layers(giver, 2, 64, 64)
    nxt, = layers(taker, 1, 64, 96)
    q.link_linears(first, nxt)
    with pytest.raises(ValueError):
        q.link_linears(second, nxt)
    assert second.y_amax_to is None
    if giver == "fp8":
        assert nxt.dx_amax_to.data_ptr() == first.sdy.amax.data_ptr()
        assert second.sdy.amax_algo != q.AMAX_PRECOMPUTED


def test_a_layer_is_linked_anew():
    """When the other one is gone, or has been given another amax_algo or no amax to deliver to."""
    import quantised_gemm_gb300 as q
    prev, = layers("fp8", 1, 64, 64)
    nxt = layers("fp8", 3, 64, 96)
    q.link_linears(prev, nxt.pop())
    q.link_linears(prev, nxt[0])
    assert prev.y_amax_to.data_ptr() == nxt[0].sx.amax.data_ptr()
    nxt[0].sx.amax_algo = q.AMAX_AUTO
    nxt[0].dx_amax_to = None
    q.link_linears(prev, nxt[1])
    assert prev.y_amax_to.data_ptr() == nxt[1].sx.amax.data_ptr()
    assert nxt[1].dx_amax_to.data_ptr() == prev.sdy.amax.data_ptr()
    norms = layers("norm", 2, 64, 0)
    lin, = layers("fp8", 1, 64, 64)
    q.link_linears(lin, norms[0])
    with pytest.raises(ValueError):
        q.link_linears(lin, norms[1])
    norms[0].dx_amax_to = None
    q.link_linears(lin, norms[1])
    assert norms[1].dx_amax_to.data_ptr() == lin.sdy.amax.data_ptr()
    by_hand, taker = layers("norm", 1, 64, 0)[0], layers("fp8", 1, 64, 96)[0]
    by_hand.y_amax_to = nxt[0].sx.amax
    with pytest.raises(ValueError):
        q.link_linears(by_hand, taker)
