"""More refusals of the windowed / paged calls and of the page calls, found on
the host before anything is enqueued (no GPU, device pointers that nothing reads)."""

import ctypes

import pytest

from test_view_refusals import INVALID, WS, ALIGNMENT, B, _pool, _table  # noqa: F401  (B is the fixture)


def test_granted_must_not_meet_lengths_or_add(B):
    L = B.load()
    a = B.tq_pages_reserve_args(_pool(B), _table(B), 0x5000, 0x6000, 0, None, 0x7000)
    for at, status in ((0x5008, INVALID), (0x5ff8, INVALID), (0x6002, ALIGNMENT)):
        a.granted = at
        assert L.tq_pages_reserve(ctypes.byref(a), WS, 1 << 40, None) == status


# ------------------------------------------------- the binding's own checks ---
def _attention(B, which, **change):
    """The arguments of a windowed / paged call on the CPU, all of them right but for the device."""
    import types

    import torch

    k, v = (B.Cache(m, 3, 128, rows=8, capacity=16, device="cpu") for m in ("prod", "mse"))
    handle = types.SimpleNamespace(handle=None)
    shape = (2, 5, 4, 128) if which == "prefill" else (2, 4, 128)
    a = dict(q=torch.zeros(shape), kcache=k, vcache=v, pos=torch.zeros(2, dtype=torch.int32), n=32, rot=handle, qjl=handle,
             out=torch.zeros(shape), k_new=torch.zeros(4, 128), v_new=torch.zeros(4, 128),
             append_pos=torch.zeros(2, dtype=torch.int32), workspace=torch.zeros(256, dtype=torch.uint8),
             view=B.View(10, 2, torch.zeros(2, 2, dtype=torch.int32), 4))
    a.update(change)
    kw = {x: a[x] for x in ("gqa_map", "logits") if x in a}
    args = [a[x] for x in ("q", "kcache", "vcache", "pos", "n", "rot", "qjl", "out")]
    if which == "step":
        args += [a["k_new"], a["v_new"], a["append_pos"]]
    fn = {"prefill": B.tq_attn_prefill_view, "decode": B.tq_attn_decode_view, "step": B.tq_decode_step_view}[which]
    return B.prepare(fn, *args, a["workspace"], a["view"], **kw)


@pytest.mark.parametrize("which", ["decode", "step", "prefill"])
def test_attention_tensors(B, which):
    """Types, shapes and strides that the kernels would read as something else, and tensors off the GPU."""
    import torch

    shape = (2, 5, 4, 128) if which == "prefill" else (2, 4, 128)
    pos = "q_start" if which == "prefill" else "seq_lens"
    wide = torch.zeros(shape[:-1] + (256,))[..., :128]
    cases = [(dict(q=wide), "q must be contiguous"), (dict(out=wide), "out must be contiguous"),
             (dict(q=torch.zeros(shape, dtype=torch.float16)), "q must be of"),
             (dict(out=torch.zeros(shape, dtype=torch.float16)), "out must be of"),
             (dict(out=torch.zeros(shape[:-1] + (64,))), "out must be contiguous and hold"),
             (dict(pos=torch.zeros(2, dtype=torch.int64)), pos), (dict(pos=torch.zeros(1, dtype=torch.int32)), pos),
             (dict(pos=torch.zeros(4, dtype=torch.int32)[::2]), pos), (dict(gqa_map=[0, 0, 1]), "gqa_map"),
             ({}, "must be on a GPU")]
    if which == "step":
        cases += [(dict(k_new=torch.zeros(4, 256)[:, :128]), "k_new must be contiguous"),
                  (dict(v_new=torch.zeros(2, 128)), "v_new must be contiguous and hold 512"),
                  (dict(v_new=torch.zeros(4, 128, dtype=torch.bfloat16)), "v_new must be of"),
                  (dict(append_pos=torch.zeros(2, dtype=torch.int64)), "append_pos")]
    if which != "prefill":
        cases += [(dict(logits=torch.zeros(2, 4, 31)), "logits must be contiguous and hold"),
                  (dict(logits=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), "logits must be of")]
    for change, message in cases:
        with pytest.raises(ValueError, match=message):
            _attention(B, which, **change)
    with pytest.raises(ValueError, match="q is on meta"):
        _attention(B, which, q=torch.zeros(shape, device="meta"))


def test_numbers_past_32_bits(B):
    import torch

    for x in ("window", "sinks", "n_pages"):
        with pytest.raises(ValueError, match=x):
            B.View(**{x: 2**32})
    k, v = (B.Cache(m, 3, 128, rows=6, capacity=16, device="cpu") for m in ("prod", "mse"))
    pool, t, n = B.PagePool(k, v, 2), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="add"):
        B.prepare(B.tq_pages_reserve, pool, t, n, 2**31, ws)
    for kw in (dict(window=2**31), dict(sinks=2**32)):
        with pytest.raises(ValueError, match="must fit 32 bits"):
            B.prepare(B.tq_pages_trim, pool, t, n, **kw)


def test_page_tensors_off_the_gpu(B):
    """Host memory never goes to a kernel: every page call refuses a pool or a tensor that is not on the GPU."""
    import torch

    k, v = (B.Cache(m, 3, 128, rows=6, capacity=16, device="cpu") for m in ("prod", "mse"))
    pool, t, n = B.PagePool(k, v, 2), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    meta = n.to("meta")
    calls = [(B.tq_pages_reserve, (pool, t, n, 1, ws)), (B.tq_pages_trim, (pool, t, n)),
             (B.tq_pages_fork, (pool, t, t.clone(), n, n, n.clone(), ws)), (B.tq_pages_copy, (pool, pool, n, n)),
             (B.tq_pages_compact, (pool, t, pool, t, ws))]
    for fn, args in calls:
        with pytest.raises(ValueError, match="must be on a GPU"):
            B.prepare(fn, *args)
        if fn is not B.tq_pages_compact:
            with pytest.raises(ValueError, match="is on meta"):
                B.prepare(fn, *(meta if x is n else x for x in args))
    with pytest.raises(ValueError, match="one device"):
        B.PagePool(k, v, 2, refs=torch.zeros(3, dtype=torch.int32, device="meta"))
