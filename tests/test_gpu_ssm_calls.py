"""The state-space block's operators as a program calls them: captured in a CUDA graph, one workspace for calls of other
sizes, calls on two streams, memory of a call on a stream that is not the current one, columns and pools beyond 32-bit
offsets. GPU only."""
import pytest

from tests import ssm_ref
from tests.test_gpu_conv_act import inputs as conv_inputs
from tests.test_gpu_ssm import int32, on_gpu, run_bwd, run_fwd
from tests.test_gpu_streams import Spy, stream_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402


def everything(d, e, **kw):
    """One call of each operator on scan inputs d and convolution inputs e."""
    n = d["x"].shape[0]
    w = d["skip"].to(d["x"].dtype)
    out, fin = gdn.ssm_scan_fwd(d["x"], d["dt"], d["a"], d["b"], d["c"], d["cu"], skip=d["skip"], z=d["z"],
                                dt_bias=d["dt_bias"], init_idx=d["idx"], initial_state=d["pool"], **kw)
    g = gdn.ssm_scan_bwd(d["x"], d["dt"], d["a"], d["b"], d["c"], d["cu"], d["dout"], dfinal_state=d["dfin"], skip=d["skip"],
                         z=d["z"], dt_bias=d["dt_bias"], init_idx=d["idx"], initial_state=d["pool"], **kw)
    y, tail = gdn.conv_fwd(e["x"], e["w"], e["cu"], bias=e["bias"], init_idx=d["idx"], conv_init=e["pool"], activation="silu", **kw)
    k = gdn.conv_bwd(e["x"], e["w"], e["cu"], e["dy"], bias=e["bias"], init_idx=d["idx"], conv_init=e["pool"],
                     dfinal_tail=e["dtail"], activation="silu", **kw)
    f = gdn.gated_rmsnorm_fwd(out, d["x"], w, group=w.shape[0] // 2, first="norm", **kw)
    dx, dz, dw = gdn.gated_rmsnorm_bwd(out, d["x"], w, d["dout"], first="gate", **kw)
    states, tails = fin.clone(), tail.clone()
    at = torch.arange(fin.shape[0], dtype=torch.int32, device="cuda") if "at" not in d else d["at"]
    m = min(n, at.shape[0])
    o = gdn.ssm_decode_step(d["x"][:m], d["dt"][:m], d["a"], d["b"][:m], d["c"][:m], states, at[:m], skip=d["skip"],
                            z=d["z"][:m], dt_bias=d["dt_bias"], **kw)
    q = gdn.conv_decode_step(e["x"][:m], e["w"], tails, at[:m], bias=e["bias"], activation="silu", **kw)
    return [out, fin, y, tail, f, dx, dz, dw, o, q, states, tails] + [v for v in list(g.values()) + list(k.values()) if v is not None]


def problem(seed, lens, C, S, G, dtype, idx=None, n_pool=1):
    d, _ = on_gpu(ssm_ref.problem(seed, lens, C, S, G, n_pool=n_pool, dfin=True), dtype)
    d["idx"] = int32(idx)
    d["at"] = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    return d, conv_inputs(seed, lens, C, dtype, n_pool=n_pool)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_captured_in_a_graph(dtype):
    d, e = problem(3, [300, 0, 700, 77], 64, 16, 2, dtype, [0, 1 + 0, -1, 1 + 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(d, e)  # attributes are set and the allocator is warm before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(d, e)
    for turn in range(2):
        for t in (d["x"], d["dout"], e["x"], e["dy"]):
            t.mul_(-0.5)  # other values in the captured places
        want = everything(d, e)
        graph.replay()
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_workspace_for_other_sizes():
    sizes = [([300, 0, 700, 77], 64, 16, 2, "bf16", [0, 1 + 0, -1, 1 + 2]), ([5], 130, 5, 1, "fp32", None),
             ([1] * 40, 24, 64, 1, "fp16", None)]
    need = max(max(gdn.ssm_workspace_size(len(n), sum(n), C, S, G, True),
                   gdn.conv_workspace_size(len(n), sum(n), C // 8 * 8, True, "silu")) for n, C, S, G, _, _ in sizes)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for lens, C, S, G, dtype, idx in sizes:
            d, _ = on_gpu(ssm_ref.problem(C, lens, C, S, G, n_pool=1, dfin=True), dtype)
            want, wantg = run_fwd(d, idx), run_bwd(d, idx)
            ws.random_(0, 256)
            got, gotg = run_fwd(d, idx, workspace=ws), run_bwd(d, idx, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(want, got)) and gdn.workspace_status(ws) == gdn.GDN_OK
            assert all(torch.equal(wantg[k], gotg[k]) for k in wantg if wantg[k] is not None)
            if C % 8:
                continue
            e = conv_inputs(C, lens, C, dtype, n_pool=1)
            kw = dict(bias=e["bias"], init_idx=int32(idx), conv_init=e["pool"], activation="silu")
            want = list(gdn.conv_fwd(e["x"], e["w"], e["cu"], **kw)) + list(gdn.conv_bwd(e["x"], e["w"], e["cu"], e["dy"], **kw).values())
            ws.random_(0, 256)
            got = list(gdn.conv_fwd(e["x"], e["w"], e["cu"], workspace=ws, **kw))
            got += list(gdn.conv_bwd(e["x"], e["w"], e["cu"], e["dy"], workspace=ws, **kw).values())
            assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_calls_on_two_streams():
    one, two = problem(5, [600, 33], 128, 16, 1, "bf16", [0, -1]), problem(6, [64, 900], 72, 8, 2, "bf16", [-1, 0])
    want = [everything(*one), everything(*two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(3):
        for i, p in enumerate((one, two)):
            with torch.cuda.stream(streams[i]):
                got[i].append(everything(*p))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], r))


NAMES = ["gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_conv_act_fwd", "gdn_conv_act_bwd", "gdn_gated_rmsnorm_fwd", "gdn_gated_rmsnorm_bwd",
         "gdn_ssm_decode_step", "gdn_conv_decode_step"]


def test_memory_of_a_call_is_its_streams(monkeypatch):
    d, e = problem(7, [500, 40], 128, 16, 1, "bf16", [0, -1])
    given = {t.data_ptr() for s in (d, e) for t in s.values() if isinstance(t, torch.Tensor)}
    given |= {t[:, :1].data_ptr() for t in (d["x"], d["dt"])}
    side, seen = torch.cuda.Stream(), []
    lib = gdn.load()
    w = d["skip"].bfloat16()
    states, tails = torch.zeros(2, 128, 16, device="cuda"), torch.zeros(2, 3, 128, dtype=torch.bfloat16, device="cuda")
    given |= {w.data_ptr(), states.data_ptr(), tails.data_ptr()}
    torch.cuda.synchronize()
    monkeypatch.setattr(gdn, "load", lambda path=None: Spy(lib, seen))
    s = dict(stream=side)
    kept = [run_fwd(d, **s), run_bwd(d, **s), gdn.conv_fwd(e["x"], e["w"], e["cu"], activation="silu", **s),
            gdn.conv_bwd(e["x"], e["w"], e["cu"], e["dy"], activation="silu", **s),
            gdn.gated_rmsnorm_fwd(d["x"], d["z"], w, **s), gdn.gated_rmsnorm_bwd(d["x"], d["z"], w, d["dout"], **s),
            gdn.ssm_decode_step(d["x"][:2], d["dt"][:2], d["a"], d["b"][:2], d["c"][:2], states, d["at"], **s),
            gdn.conv_decode_step(e["x"][:2], e["w"], tails, d["at"], **s)]
    side.synchronize()
    made = {a for a in seen if a != side.cuda_stream and a not in given}
    assert len(kept) == len(NAMES) and len(made) >= 12 and all(stream_of(a) == side.cuda_stream for a in made)


def test_pools_beyond_32_bit_offsets():
    """Entries whose first element lies more than 2^32 bytes (the states) and 2^31 elements (the tails) into the pool."""
    C, S = 4096, 64
    n = (1 << 31) // (C * S) + 2  # 8.6 GB of states
    pool = torch.zeros(n, C, S, device="cuda")
    pool[n - 1] = torch.randn(C, S, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    d, _ = on_gpu(ssm_ref.problem(9, [3], C, S), "bf16")
    small = pool[n - 1:].clone()
    d["pool"] = small
    want, wfin = run_fwd(d, [0])
    d["pool"] = pool
    out, fin = run_fwd(d, [n - 1])
    assert torch.equal(out, want) and torch.equal(fin, wfin)
    one = {k: d[k][:1] for k in ("x", "dt", "z", "b", "c")}
    step = lambda p, i: gdn.ssm_decode_step(one["x"], one["dt"], d["a"], one["b"], one["c"], p, int32([i]), skip=d["skip"],  # noqa: E731
                                            z=one["z"], dt_bias=d["dt_bias"])
    assert torch.equal(step(small, 0), step(pool, n - 1)) and torch.equal(small[0], pool[n - 1])
    assert not pool[:n - 1].any()
    del pool
    C = 1 << 16
    n = (1 << 31) // (3 * C) + 2  # 4.3 GB of tails
    tails = torch.zeros(n, 3, C, dtype=torch.bfloat16, device="cuda")
    tails[n - 1] = 1.5
    x, w = torch.ones(1, C, dtype=torch.bfloat16, device="cuda"), torch.rand(C, 4, device="cuda")
    small = tails[n - 1:].clone()
    assert torch.equal(gdn.conv_decode_step(x, w, small, int32([0])), gdn.conv_decode_step(x, w, tails, int32([n - 1])))
    assert torch.equal(small[0], tails[n - 1]) and not tails[:n - 1].any()


def test_rows_beyond_32_bit_offsets():
    """The last rows of tensors of more than 2^31 elements, against the same rows by themselves."""
    T, D = 70000, 32768
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x[-40:] = torch.randn(40, D, device="cuda", generator=gen).bfloat16()
    w = torch.rand(128, device="cuda", generator=gen).bfloat16()
    y = gdn.gated_rmsnorm_fwd(x, x, w, group=128)
    assert torch.equal(y[-40:], gdn.gated_rmsnorm_fwd(x[-40:], x[-40:], w, group=128)) and not y[:-40].any()
    dx, dz, dw = gdn.gated_rmsnorm_bwd(x, x, w, x, group=128)
    a, b, c = gdn.gated_rmsnorm_bwd(x[-40:], x[-40:], w, x[-40:], group=128)
    assert torch.equal(dx[-40:], a) and torch.equal(dz[-40:], b)
    torch.testing.assert_close(dw, c, rtol=40 * 256 * 2.0 ** -24, atol=float(c.abs().max()) * 40 * 256 * 2.0 ** -24)
    del y, dx, dz
    taps = torch.rand(D, 4, device="cuda", generator=gen)
    cu = int32([0, T - 40, T])
    y, tail = gdn.conv_fwd(x, taps, cu, activation="silu")
    ys, ts = gdn.conv_fwd(x[-40:], taps, int32([0, 40]), activation="silu")
    assert torch.equal(y[-40:], ys) and torch.equal(tail[1], ts[0])
    del y
    g = gdn.conv_bwd(x, taps, cu, x, activation="silu")
    gs = gdn.conv_bwd(x[-40:], taps, int32([0, 40]), x[-40:], activation="silu")
    torch.testing.assert_close(g["dx"][-40:], gs["dx"], rtol=2.0 ** -20, atol=float(gs["dx"].abs().max()) * 2.0 ** -20)
    del g
    a_, b = -torch.rand(D, 2, device="cuda", generator=gen), torch.ones(T, 1, 2, dtype=torch.bfloat16, device="cuda")
    out, fin = gdn.ssm_scan_fwd(x, x, a_, b, b, cu)
    os_, fs = gdn.ssm_scan_fwd(x[-40:], x[-40:], a_, b[-40:], b[-40:], int32([0, 40]))
    near = dict(rtol=2.0 ** -7, atol=float(os_.abs().max()) * 2.0 ** -14)  # other segments: a rounding to bf16 may turn
    torch.testing.assert_close(out[-40:], os_, **near)
    torch.testing.assert_close(fin[1], fs[0], rtol=2.0 ** -14, atol=2.0 ** -14)


def test_pools_of_many_entries():
    """Thousands of documents, each from an entry of its own or from one that many share: gradients against those of the
    documents by themselves, and the time stays that of the sizes."""
    N, C, S = 6000, 24, 8
    rng = torch.Generator().manual_seed(5)
    own = torch.randperm(N, generator=rng)
    own[::3] = 7
    lens = [1] * N
    d, _ = on_gpu(ssm_ref.problem(8, lens, C, S, n_pool=1, dfin=True), "fp32")
    d["pool"] = torch.randn(N, C, S, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    g = run_bwd(d, own.tolist())
    alone = run_bwd(d | {"pool": d["pool"][own.to("cuda")].contiguous()}, list(range(N)))
    want = torch.zeros(N, C, S, dtype=torch.float64, device="cuda").index_add_(0, own.to("cuda"), alone["dinit"].double())
    torch.testing.assert_close(g["dinit"].double(), want, rtol=2.0 ** -20, atol=2000 * 2.0 ** -24 * float(want.abs().max()))
    e = conv_inputs(9, lens, C, "fp32")
    pool = torch.randn(N, 3, C, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    run = lambda p, i: gdn.conv_bwd(e["x"], e["w"], e["cu"], e["dy"], bias=e["bias"], init_idx=int32(i), conv_init=p,  # noqa: E731
                                    dfinal_tail=e["dtail"], activation="silu")["dconv_init"]
    got, alone = run(pool, own.tolist()), run(pool[own.to("cuda")].contiguous(), list(range(N)))
    want = torch.zeros(N, 3, C, dtype=torch.float64, device="cuda").index_add_(0, own.to("cuda"), alone.double())
    torch.testing.assert_close(got.double(), want, rtol=2.0 ** -20, atol=2000 * 2.0 ** -24 * float(want.abs().max()))


def test_a_document_of_almost_the_most_tokens():
    """One channel and a document so long that its last segment's end, in whole tiles, lies beyond 31 bits. Tokens of zeros
    have a step of zero, so they leave the state: what the others make of it, from the first segment to the last, is the
    same as in a document of those alone."""
    torch.cuda.empty_cache()
    T = 2 ** 31 - 5000
    if torch.cuda.mem_get_info()[0] < gdn.ssm_workspace_size(1, T, 1, 1) + (12 << 30):
        pytest.skip("needs 160 GB of free memory")
    marks = torch.tensor([0, 1, 20, 883023, 883024, T // 2, T - 900000, T - 883024, T - 3, T - 2, T - 1], device="cuda")
    values = torch.linspace(0.2, 1.0, len(marks), device="cuda").bfloat16().unsqueeze(1)
    v = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    v[marks] = values
    a = torch.tensor([[-0.5]], device="cuda")
    run = lambda x, **kw: gdn.ssm_scan_fwd(x, x, a, x.unsqueeze(2), x.unsqueeze(2), int32([0, x.shape[0]]),  # noqa: E731
                                           dt_softplus=False, **kw)
    want, wfin = run(values)
    out = torch.full((T, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gdn.ssm_workspace_size(1, T, 1, 1), dtype=torch.uint8, device="cuda")
    _, fin = run(v, out=out, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    got = out[marks].clone()
    # each token's step rounds as often as in the short document (2^-21 a token); a state that is carried over a segment
    # of zeros alone is multiplied by exp(0) = 1; an output rounded to bf16 may turn (2^-8 of it on either side)
    torch.testing.assert_close(fin, wfin, rtol=len(marks) * 2.0 ** -20, atol=0)
    torch.testing.assert_close(got.float(), want.float(), rtol=2.0 ** -7, atol=0)
    out[marks] = 0
    assert not out.any()
    del v, out, ws
    torch.cuda.empty_cache()
