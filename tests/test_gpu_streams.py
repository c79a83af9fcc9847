"""Calls on a stream that is not the current one (stream=...): the memory that a call allocates for itself belongs to
the stream it runs on. If it came from the current stream's share of the allocator's cache, the current stream could
be given the workspace again while the call still runs, or the call could be given memory that the current stream is
still writing. GPU only: addresses are compared, nothing is run at the same time."""
import pytest

import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402


class Spy:
    """The library, with a note of each call's pointers."""

    def __init__(self, lib, seen):
        self.lib, self.seen = lib, seen

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if name.endswith("_size"):
            return fn

        def call(*args):
            self.seen += [a for a in args if isinstance(a, int) and a > 1 << 32]
            return fn(*args)
        return call


def calls():
    """Each call as a function of its stream, and the addresses of all inputs."""
    T = 2048
    d = synth.to_device(synth.make_problem("streams", 61, [T - 300, 300], 2, 4, with_dout=True))
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do, cu, gate, beta = (d[x] for x in ("q", "k", "v", "dout", "cu_seqlens", "g", "beta"))
    g = -torch.rand(4, generator=gen, device="cuda")
    pool, idx = rand(64, 4, 128, 128), torch.arange(64, dtype=torch.int32, device="cuda")
    x, w, taps, bias = rand(T, 1024).bfloat16(), rand(1024).bfloat16(), rand(1024, 4), rand(1024)
    inputs = {t.data_ptr() for t in (q, k, v, do, cu, gate, beta, g, pool, idx, x, w, taps, bias)}
    return inputs, dict(
        chunk_fwd=lambda **s: gdn.chunk_fwd(q, k, v, gate, beta, cu, **s),
        chunk_bwd=lambda **s: gdn.chunk_bwd(q, k, v, gate, beta, cu, do, **s),
        decode_step=lambda **s: gdn.decode_step(q[:64], k[:64], v[:64], gate[:64], beta[:64], pool, idx, **s),
        conv_fwd=lambda **s: gdn.conv_fwd(x, taps, cu, **s),
        conv_bwd=lambda **s: gdn.conv_bwd(x, taps, cu, x, bias=bias, **s),
        la_chunk_fwd=lambda **s: gdn.la_chunk_fwd(q, k, v, g, cu, **s),
        la_chunk_bwd=lambda **s: gdn.la_chunk_bwd(q, k, v, g, cu, do, **s),
        la_decode_step=lambda **s: gdn.la_decode_step(q[:64], k[:64], v[:64], g, pool, idx, **s),
        rmsnorm_fwd=lambda **s: gdn.rmsnorm_fwd(x, w, residual=x, quant="group", **s),
        rmsnorm_bwd=lambda **s: gdn.rmsnorm_bwd(x, w, x, **s))


def stream_of(address):
    for b in torch.cuda.memory_snapshot():
        if b["address"] <= address < b["address"] + b["total_size"]:
            return b["stream"]
    raise AssertionError("not memory of the allocator")


@pytest.mark.parametrize("name", ["chunk_fwd", "chunk_bwd", "decode_step", "conv_fwd", "conv_bwd", "la_chunk_fwd",
                                  "la_chunk_bwd", "la_decode_step", "rmsnorm_fwd", "rmsnorm_bwd"])
def test_memory_of_a_call_is_its_streams(name, monkeypatch):
    inputs, call = calls()
    side, seen = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    monkeypatch.setattr(gdn, "load", lambda path=None, lib=gdn.load(): Spy(lib, seen))
    kept = call[name](stream=side)
    side.synchronize()
    made = {a for a in seen if a != side.cuda_stream and a not in inputs}  # outputs and workspace
    assert made and all(stream_of(a) == side.cuda_stream for a in made)
    del kept
