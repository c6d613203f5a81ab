"""Calls that overlap others: chained on one stream, and on streams of several threads.

The block-scaled products start as programmatic dependents of the quantisation that
writes their operands and scales, and must read neither before it has ended. Each chain
writes the same buffers again with other data, with nothing in between that waits, and
every result has the bits of calls that wait for each other."""
import threading

import pytest
import torch

from dense_gemm_row_gb300.feed_forward import FeedForward, GatedFeedForward
from tests.layer_util import normal

pytestmark = pytest.mark.gpu

# Tokens, outputs and k: both few-rows forms and both tile widths, one k-block and more
# than the kernels have in flight, and scales in rows off 16-byte boundaries.
SHAPES = [(1, 1024, 512), (20, 4096, 2048), (64, 640, 4096), (300, 264, 136), (700, 2048, 1024),
          (1100, 4096, 1152)]


def empty(rows, cols, block_rows):
    ld = -(-cols // 16) * 16
    return (torch.zeros(rows, ld, dtype=torch.float8_e4m3fn, device="cuda")[:, :cols],
            torch.zeros(-(-rows // block_rows), -(-cols // 128), device="cuda"))


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_quantise_then_product_into_the_same_buffers(gemm_mod, shape, gated):
    g, dtype, reps = gemm_mod, torch.bfloat16, 6
    m, n, k = shape
    # Sizes a factor of 16 apart from one repetition to the next: a scale that is not the
    # repetition's own shows in every value that it touches.
    xs = [normal((m, k), dtype, i, 16.0 ** (i % 3)) for i in range(reps)]
    ws = [normal((n, k), dtype, 50 + i, 16.0 ** -(i % 2)) for i in range(reps)]
    us = [normal((n, k), dtype, 90 + i, 16.0 ** ((i + 1) % 2)) for i in range(reps)]
    (a, sa), (b, sb), (u, su) = empty(m, k, 1), empty(n, k, 128), empty(n, k, 128)

    def run(wait):
        outs = []
        for x, w, v in zip(xs, ws, us):
            D = torch.empty(m, n, dtype=dtype, device="cuda")
            steps = [lambda: g.quantise_blocks(w, b, sb, rows=128)]
            if gated:
                steps += [lambda: g.quantise_blocks(v, u, su, rows=128),
                          lambda: g.quantise_blocks(x, a, sa),
                          lambda: g.gemm_gated(a, b, u, D, act="none", trans_b=True, scale_a=sa,
                                               scale_gate=sb, scale_up=su)]
            else:
                steps += [lambda: g.quantise_blocks(x, a, sa),
                          lambda: g.gemm_epilogue(a, b, D, trans_b=True, scale_a=sa, scale_b=sb)]
            for step in steps:
                step()
                if wait:
                    torch.cuda.synchronize()
            outs.append(D)
        return outs

    want = run(True)
    for _ in range(3):
        got = run(False)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(bool(p.isfinite().all()) for p in want)
    assert g.check_device_error() == 0


def test_steps_of_several_threads_at_once(gemm_mod):
    """Training steps and 8-bit passes on four threads' streams: the bits of each alone."""
    def job(seed, tokens, model, hidden, kind):
        ff = kind(model, hidden, "silu", seed=seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x, r, dout = (torch.randn(tokens, model, generator=gen, device="cuda").bfloat16()
                      for _ in range(3))

        def step():
            out, saved = ff.forward(x, r)
            return [out, ff.forward8(x, r), *ff.backward(dout, saved).values()]
        return step

    jobs = [job(1, 300, 512, 1040, GatedFeedForward), job(2, 7, 1024, 2048, GatedFeedForward),
            job(3, 1500, 256, 800, GatedFeedForward), job(4, 100, 512, 1024, FeedForward)]
    want = [step() for step in jobs]
    torch.cuda.synchronize()
    done, wrong = [], []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for rep in range(20):
                got = jobs[i]()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append((i, rep))
        done.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert sorted(done) == list(range(len(jobs))) and not wrong
    assert gemm_mod.check_device_error() == 0
