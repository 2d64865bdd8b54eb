"""Refusals of the block-scaled calls' binding beside those of the library, on the CPU."""
import pytest
import torch


def _tensors():
    s, kc = torch.zeros(4, 2), torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    return (torch.zeros(3, 2, 64, dtype=torch.bfloat16), kc, s, torch.zeros(3, 1, dtype=torch.int32),
            torch.zeros(3, dtype=torch.int32))


def test_plan_refuses_shapes_like_the_call(pkv_lib):
    """Tensors of another rank: the call's own error, not one of the plan's on its way to a workspace."""
    q, kc, s, tables, lens = _tensors()
    for kw in (dict(q=q[0]), dict(tables=tables[:, 0]), dict(kc=kc[0]), dict(lens=lens[:2])):
        a = dict(q=q, kc=kc, tables=tables, lens=lens)
        a.update(kw)
        with pytest.raises(ValueError, match="paged_attention_decode_scaled"):
            pkv_lib.paged_attention_decode_scaled(a["q"], a["kc"], a["kc"], s, s, a["tables"], a["lens"], 0.1)
        with pytest.raises(ValueError, match="paged_attention_decode_scaled"):
            pkv_lib.DecodePlan(a["q"], a["kc"], a["kc"], a["tables"], a["lens"], 0.1, k_scales=s, v_scales=s)


def test_plan_runs_on_its_tensors_device(pkv_lib, monkeypatch):
    """The device is the tensors', whichever is current; it is current again afterwards."""
    current, at = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    plan = object.__new__(pkv_lib.DecodePlan)
    plan.func, plan.out, plan._args, plan._device = "paged_attention_decode_scaled", None, (), torch.device("cuda", 1)
    plan._fn = lambda *args: at.append(current[0]) or 0
    plan.run()
    assert at == [1] and current == [0]
    current[0] = 1
    plan.run()
    assert at == [1, 1]


def test_cache_refuses_half_a_pair_of_scales(pkv_lib):
    """One kind of scales given: the other's pool would be read with scales of zero."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    for kw in (dict(k_scales=torch.ones(4, 2)), dict(v_scales=torch.ones(4, 2), block_scales=True)):
        with pytest.raises(ValueError, match="go together"):
            PagedKVCache(4, 2, 16, 64, device="cpu", **kw)


def test_extend_refuses_buffers_that_overlap(pkv_lib):
    """Every written buffer against every other one, by a few bytes; lengths and head may be updated in place.  (The
    slots' alignment is refused after the overlaps, so that no call is enqueued.)"""
    lib = pkv_lib._native.lib()
    B, T, max_blocks, free = 5, 7, 3, 9
    sizes = dict(tables=4 * B * max_blocks, ctx=4 * B, new=4 * B, free=4 * free, head=4, slots=8 * T, pos=4 * T,
                 ss=4 * (B + 1), bst=4 * (B + 1), lens=4 * B, hout=4)
    apart = {name: 0x10000 + 0x1000 * i + 8 * (name == "slots") for i, name in enumerate(sizes)}

    def refusal(**kw):
        a = {**apart, **kw}
        code = lib.paged_extend_tables(a["tables"], max_blocks, a["ctx"], a["new"], B, 16, a["free"], free, a["head"],
                                       64, T, a["slots"], a["pos"], a["ss"], a["bst"], a["lens"], a["hout"], None)
        assert code == pkv_lib.ERR_INVALID
        return lib.pkv_last_error().decode()

    assert "16-byte aligned" in refusal()
    assert "16-byte aligned" in refusal(lens=apart["ctx"], hout=apart["head"])
    assert "16-byte aligned" in refusal(ctx=apart["new"], head=apart["free"])  # both read
    assert "16-byte aligned" in refusal(bst=apart["ss"] + sizes["ss"])         # next to one another
    written = ("tables", "slots", "pos", "ss", "bst", "lens", "hout")
    for w in written:
        for other in sizes:
            if other == w or (w, other) in (("lens", "ctx"), ("hout", "head")):
                continue
            assert "buffers of their own" in refusal(**{w: apart[other] + sizes[other] - 4}), (w, other)
            assert "buffers of their own" in refusal(**{w: apart[other]}), (w, other)
    assert "buffers of their own" in refusal(lens=apart["ctx"] + 4)


def test_rope_append_refuses_queries_written_over_its_inputs(pkv_lib):
    """q_out over other rows of q, over k or over v.  Beside them in one buffer it is let through, up to the refusal of
    the cache's alignment, which comes last, so that no call is enqueued."""
    lib = pkv_lib._native.lib()
    A, T, hq, hkv, D = 1 << 20, 5, 4, 2, 64
    row = (hq + 2 * hkv) * D  # one projection's output: [q | k | v]
    K, V, far = A + 2 * hq * D, A + 2 * (hq + hkv) * D, A + (1 << 16)

    def refusal(q=A, qs=row, k=K, ks=row, v=V, vs=row, qo=A, qos=row, T=T):
        code = lib.paged_rope_append(q, qs, k, ks, v, vs, A, A, T, A, D, 0, 1.0, qo, qos, far + 2, far, 8, hq, hkv, 16,
                                     D, 1, 1, None, None, None, None, None)
        assert code == pkv_lib.ERR_INVALID
        return lib.pkv_last_error().decode()

    for ok in (dict(), dict(qo=far), dict(qo=far, qs=0, ks=0, vs=0), dict(qo=A + 2 * row * T),
               dict(T=1, qo=K + 2 * row), dict(q=far, qo=A),
               dict(q=A, qo=A + 2 * row, qos=2 * row, k=far, v=far, qs=2 * row)):
        assert "16-byte aligned" in refusal(**ok), ok
    for bad in (dict(qo=K), dict(qo=V), dict(qo=A + 16), dict(qo=A + 2 * row), dict(qo=A - 2 * row), dict(qo=K - 16),
                dict(q=far, qo=A, qos=2 * row), dict(q=far, qo=V + 2 * hkv * D - 16), dict(q=far, qo=A, k=A, ks=0),
                dict(T=1, qo=K), dict(T=1, qo=A + 16)):
        assert "shares no memory" in refusal(**bad), bad
