"""GPU: what calls of the 8-bit operators leave to their caller and what they do not: kernels before
them that take long, streams, defaults, threads."""
from __future__ import annotations

import threading
import time

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from tests import test_gpu_lm as T  # noqa: E402

SYNC = V.VOC_FLAG_SYNC


# ------------------------------------------------------------------ a long kernel in front
@pytest.mark.parametrize("m,n", [(8, 1536), (2100, 1100)])
def test_linear_behind_a_kernel_of_seconds(m, n):
    """A product starts beside the kernel before it where that leaves SMs free.  Its waits' limit
    (about 2 s) counts from that kernel's end: here an attention of about 3 s on 80 SMs, over caches
    whose blocks are all one page."""
    k, seqs, rows = 1000, 80, 200
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = T._codes(g, m, k), T._codes(g, n, k)
    xs, ws = torch.rand(m, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    ref = V.linear_fp8(x, xs, w, ws, flags=SYNC)
    cache = V.KVCacheFP8.empty(1, 1, 64)
    q = torch.zeros(seqs * rows, 1, 64, dtype=torch.bfloat16, device="cuda")

    def attend(table, blocks):
        lens = torch.full((seqs,), 64 * blocks, dtype=torch.int32, device="cuda")
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        marks[0].record()
        V.attention_fp8(q, cache, table, lens, max_q=rows)
        marks[1].record()
        return marks

    def seconds(marks):
        torch.cuda.synchronize()
        return marks[0].elapsed_time(marks[1]) / 1e3

    few = 20000
    table = torch.zeros(seqs, few, dtype=torch.int32, device="cuda")
    attend(table, few)
    blocks = min(int(few * 3 / seconds(attend(table, few))), 5_000_000)
    table = torch.zeros(seqs, blocks, dtype=torch.int32, device="cuda")
    marks = attend(table, blocks)
    y = V.linear_fp8(x, xs, w, ws)
    assert 2.2 < seconds(marks) < 6
    assert torch.equal(y, ref)
    V.linear_fp8(x, xs, w, ws, flags=SYNC)  # would report a wait that gave up


# ------------------------------------------------------------------ lengths made just before
@pytest.mark.parametrize("heads,rows", [(4, 1), (2, 40)])
def test_attention_takes_lengths_of_the_kernel_in_front(heads, rows):
    """Lengths (and with them the shares of the CTAs and the parts that are joined) that change from
    call to call, written right in front of the call, against the same lengths at rest."""
    seqs, cols = 3, 130
    bt = T.Batch([64 * cols] * seqs, [rows] * seqs, 1, 64, seed=rows, spare_cols=0)
    q = T._queries(bt, heads)
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(rows, 64 * cols + 1, (40, seqs), generator=g, dtype=torch.int32).cuda()
    place = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = []
    for row in lens:
        place.copy_(row)
        got.append(V.attention_fp8(q, bt.cache, bt.t_table, place, max_q=rows))
    torch.cuda.synchronize()
    for row, o in zip(lens, got):
        assert torch.equal(V.attention_fp8(q, bt.cache, bt.t_table, row.clone(), max_q=rows, flags=SYNC), o)


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("op", ["rows", "linear", "attention"])
def test_given_stream_leaves_memory_that_the_current_one_still_reads(op):
    """A tensor whose last read waits in the current stream's queue is dropped, and a call on another
    stream gets its memory for a result: the read still finds the old values."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(64, 2048, generator=g, device="cuda").bfloat16()
    w = torch.ones(2048, device="cuda").bfloat16()
    x8, xs, _ = V.rows_fp8(x, V.VOC_LM_NONE)
    bt = T.Batch([300] * 64, [1] * 64, 2, 64, seed=1)
    q = T._queries(bt, 4)
    calls = dict(
        rows=(lambda **kw: V.rows_fp8(x, weight=w, residual=x, **kw), 64 * 2048 * 2),
        linear=(lambda **kw: (V.linear_fp8(x8, xs, x8, xs, **kw),), 64 * 64 * 2),
        attention=(lambda **kw: (V.attention_fp8(q, bt.cache, **bt.args(), **kw),), 64 * 4 * 64 * 2))
    call, size = calls[op]
    ref = call()  # set-up, and the result
    ref = [t.clone() for t in ref]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full((size,), 77, dtype=torch.uint8, device="cuda")
    kept = torch.empty_like(old)
    torch.cuda.synchronize()
    where = old.data_ptr()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    kept.copy_(old)
    del old
    got = call(stream=side)
    torch.cuda.synchronize()
    assert where in [t.data_ptr() for t in got]
    assert torch.all(kept == 77)
    for a, b in zip(got, ref):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ defaults
@pytest.mark.parametrize("lens,new", [([300, 64, 90], [17, 64, 1]), ([5, 700], [1, 0]),
                                      ([70, 1, 128], [1, 1, 1])])
def test_sequences_of_any_number_of_tokens_without_max_q(lens, new):
    """With cu_q every new token is stored and attended to, whether or not max_q is given."""
    a, b = (T.Batch(lens, new, 2, 64, seed=3, filled=False) for _ in range(2))
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    k, v = (torch.from_numpy(a.rng.standard_normal((a.total, 2, 64))).cuda().bfloat16()
            for _ in range(2))
    q = T._queries(a, 4)
    batch = dict(page_table=a.t_table, kv_lens=a.t_lens, cu_q=cu)
    V.kv_append_fp8(a.cache, k, v, flags=SYNC, **batch)
    V.kv_append_fp8(b.cache, k, v, flags=SYNC, max_q=max(new), **batch)
    for name in ("k", "v", "k_scale", "v_scale"):
        x, y = (getattr(t.cache, name).view(torch.uint8) for t in (a, b))
        assert torch.equal(x, y)
    T.R.append(a.kc, a.vc, a.ks, a.vs, T._np(k), T._np(v), a.table, lens, new)
    o = V.attention_fp8(q, a.cache, flags=SYNC, **batch)
    ref, mag, s = T.R.attention(T._np(q), a.kc, a.vc, a.ks, a.vs, a.table, lens, new, 0.125)
    rel = 2.0 ** -11 + 2.0 ** -16 + 2 * 1.5 * 64 * 2.0 ** -24 * s
    tol = rel[..., None] * mag + T.UNIT[q.dtype] * abs(ref) + 2.0 ** -30
    assert (abs(T._np(o) - ref) <= tol).all()


def test_one_token_each_is_the_default_without_cu_q():
    bt = T.Batch([70, 3], [1, 1], 1, 64)
    q = T._queries(bt, 2)
    batch = dict(page_table=bt.t_table, kv_lens=bt.t_lens)
    assert torch.equal(V.attention_fp8(q, bt.cache, flags=SYNC, **batch),
                       V.attention_fp8(q, bt.cache, max_q=1, flags=SYNC, **batch))
    with pytest.raises(V.VocoderError) as e:
        V.attention_fp8(torch.cat([q, q]), bt.cache, **batch)
    assert e.value.status == V.VOC_INVALID_ARG


# ------------------------------------------------------------------ threads
@pytest.mark.parametrize("op", ["rows", "linear", "append", "attention"])
def test_other_threads_run_while_a_call_waits_for_its_stream(op):
    """A call with VOC_FLAG_SYNC behind half a second of work: the interpreter stays free."""
    x = torch.randn(4, 256, device="cuda").bfloat16()
    x8, xs, _ = V.rows_fp8(x, V.VOC_LM_NONE)
    bt = T.Batch([70, 9], [1, 1], 2, 64)
    q = T._queries(bt, 4)
    k = torch.zeros(2, 2, 64, device="cuda").bfloat16()
    call = dict(rows=lambda: V.rows_fp8(x, V.VOC_LM_NONE, flags=SYNC),
                linear=lambda: V.linear_fp8(x8, xs, x8, xs, flags=SYNC),
                append=lambda: V.kv_append_fp8(bt.cache, k, k, flags=SYNC, **bt.args()),
                attention=lambda: V.attention_fp8(q, bt.cache, flags=SYNC, **bt.args()))[op]
    call()
    waited = []

    def wait():
        torch.cuda._sleep(1_000_000_000)
        start = time.perf_counter()
        call()
        waited.append(time.perf_counter() - start)

    thread = threading.Thread(target=wait)
    thread.start()
    last, gap = time.perf_counter(), 0.0
    while thread.is_alive():
        time.sleep(0.005)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    assert waited and waited[0] > 0.25
    assert gap < 0.2
