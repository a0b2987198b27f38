"""Calls of several host threads at once, each on its own stream: kernels whose shared memory
depends on the call must not be refused because another thread has just prepared the same
kernel for less."""
import threading

import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from state_space_model_chunked_gb300._binding import load

pytestmark = pytest.mark.gpu


def at_once(*calls, times=6000):
    """Each of `calls`, given a stream, that many times on a thread of its own; what went wrong."""
    errors, start = [], threading.Barrier(len(calls))

    def work(call):
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()) as _:
            stream = torch.cuda.current_stream().cuda_stream
            start.wait()
            try:
                for _ in range(times):
                    status = call(stream)
                    if isinstance(status, int) and status:
                        raise RuntimeError(f"status {status}")
            except Exception as e:     # noqa: BLE001
                errors.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def test_embedding_gradients_of_few_and_many_tokens():
    vocab, width, lib = 600, 8, load()
    made = []
    for count in (300, 30000, 90000):
        gen = torch.Generator(device="cuda").manual_seed(count)
        t = torch.randint(vocab, (count,), device="cuda", generator=gen)
        dy = torch.randn((count, width), device="cuda", generator=gen)
        want = ssd.embedding_bwd(dy, t, vocab)
        out, need = torch.empty_like(want), ssd.embedding_bwd_workspace_bytes(count, vocab, width)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        args = (dy.data_ptr(), t.data_ptr(), 1, 0, 0, count, vocab, width, width, 1.0, out.data_ptr(), ws.data_ptr(), need)
        made.append((lambda s, args=args: lib.ssd_embedding_bwd(*args, s), out, want, (dy, t, ws)))
    assert at_once(*(call for call, *_ in made)) == []
    assert all(torch.equal(out, want) for _, out, want, _ in made)


def test_layer_norms_of_narrow_and_wide_rows():
    made, lib = [], load()
    for width, residual in ((1544, False), (1544, True), (1800, False), (2048, True)):      # one kernel: 8 runs a lane
        gen = torch.Generator(device="cuda").manual_seed(width)
        x = torch.randn((2500, width), device="cuda", generator=gen).bfloat16()
        w, r = torch.randn((width,), device="cuda", generator=gen), x * 2
        want = ssd.layernorm_fwd(x, w, None, r if residual else None, out_dtype=torch.float8_e4m3fn)
        y, so, mean, rstd, scale = (torch.empty_like(t) for t in (want[0], r, *want[2:]))
        args = (x.data_ptr(), r.data_ptr() if residual else None, w.data_ptr(), None, 1e-5, 1, 1, 2, 2500, width, width, width,
                y.data_ptr(), so.data_ptr(), mean.data_ptr(), rstd.data_ptr(), scale.data_ptr())
        made.append((lambda s, args=args: lib.ssd_layernorm_fwd(*args, s), y, scale, want, (x, w, r, so, mean, rstd)))
    assert at_once(*(call for call, *_ in made)) == []
    for _, y, scale, want, _ in made:
        assert torch.equal(y.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scale, want[4])


def test_single_tokens_and_scans_of_several_state_sizes():
    """The decode kernels' shared memory goes by the head's rows, the fp32 scan's by the state's
    columns."""
    made = []
    dev = dict(device="cuda")
    for heads, p, n, tokens in ((8, 16, 128, 4), (8, 64, 128, 4), (8, 64, 128, 1), (8, 128, 128, 1)):
        batch = 160                     # the streaming kernel's number of states
        lead = (batch, tokens) if tokens > 1 else (batch,)
        state, D = torch.zeros((batch, heads, p, n), **dev), torch.zeros(heads, **dev)
        x, dt = torch.randn((*lead, heads, p), **dev), torch.rand((*lead, heads), **dev)
        A, B, C = -torch.ones(heads, **dev), torch.randn((*lead, 1, n), **dev), torch.randn((*lead, 1, n), **dev)
        run = ssd.state_update_multi if tokens > 1 else ssd.state_update
        made.append(lambda _, run=run, a=(state, x, dt, A, B, C, D): run(*a))
    for n in (16, 256):
        x, dt, A = torch.randn((1, 64, 1, 16), **dev), torch.rand((1, 64, 1), **dev), -torch.ones(1, **dev)
        B, C = torch.randn((1, 64, 1, n), **dev), torch.randn((1, 64, 1, n), **dev)
        made.append(lambda _, a=(x, dt, A, B, C): ssd.scan_fwd(*a))
    assert at_once(*made, times=2000) == []


def test_delta_rules_of_several_streams_side_by_side():
    """Kernels that take an SM's tensor memory, and others, of calls in flight at once: equal bits."""
    made = []
    unit = torch.nn.functional.normalize
    for seed, (nseq, length, groups, heads, p, n, dtype) in enumerate(((1, 3300, 1, 2, 64, 64, torch.bfloat16), (3, 500, 2, 4, 128, 128, torch.bfloat16),
                                                                       (2, 300, 1, 2, 60, 100, torch.bfloat16), (5, 200, 2, 2, 64, 128, torch.float32))):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(s, device="cuda", generator=gen)   # noqa: E731
        x = [unit(new(nseq, length, groups, n), dim=-1).to(dtype), unit(new(nseq, length, groups, n), dim=-1).to(dtype),
             new(nseq, length, heads, p).to(dtype), -0.1 * new(nseq, length, heads).abs(), new(nseq, length, heads).sigmoid()]
        do = new(nseq, length, heads, p).to(dtype)
        w, wide = new(256, 512).bfloat16(), new(4096, 512).bfloat16()

        def call(_, x=x, do=do, w=w, wide=wide, last=None):
            o, final, kept = ssd.delta_scan_fwd(*x, return_checkpoints=True)
            last[:] = [o, final, *ssd.delta_scan_bwd(do, *x, kept), ssd.linear_fwd(wide, w)]
        want, last = [], []
        call(None, last=want)
        made.append((lambda s, call=call, last=last: call(s, last=last), last, want))
    assert at_once(*(call for call, _, _ in made), times=150) == []
    for _, last, want in made:
        assert all(torch.equal(a, b) for a, b in zip(last, want))
