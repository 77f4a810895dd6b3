"""Calls that take the tensor-core kernel beside own rows (asserted, not assumed), and calls from two threads at once."""
import threading

import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
from attention_paths import make, prefix_kernel  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [0, 5, 90])
@pytest.mark.parametrize("B,N,H,D,P", [(128, 1, 8, 128, 190), (2, 40, 2, 128, 17000), (3, 12, 2, 64, 66001), (33, 4, 8, 128, 801),
                                       (70, 8, 2, 128, 1400), (33, 4, 2, 64, 6000), (200, 2, 1, 128, 1000), (16, 12, 2, 64, 13000)])
def test_own_rows_beside_the_prefix_kernel(kvx, B, N, H, D, P, n, dtype):
    """Equal lengths, then unequal ones with none among them and NaN past the longest."""
    q, rows = make(B, N, H, D, n=n, P=P, new=n != 5, dtype=dtype, seed=P + n)
    assert prefix_kernel(kvx, q, **rows)
    ref.check_attend(kvx, q, **rows)
    gen = torch.Generator().manual_seed(P)
    extra = {"prefix_lens": torch.randint(0, P - 60, (B,), dtype=torch.int32, generator=gen).cuda()}
    extra["prefix_lens"][B // 3:B // 2] = 0
    top = int(extra["prefix_lens"].max())
    rows["prefix_k"][:, top:], rows["prefix_v"][:, top:] = float("nan"), float("nan")
    if n:
        extra["lens"] = torch.randint(0, n + 1, (B,), dtype=torch.int32, generator=gen).cuda()
        extra["lens"][B // 4:B // 2 + 1] = 0
    ref.check_attend(kvx, q, **extra, **rows)


def test_two_threads_at_once(kvx):
    """Each thread on its own stream with its own calls (another frequency table, other kernels): the bits of the calls
    made one after the other."""
    jobs = []
    for i, (theta, D, dtype) in enumerate([(1e4, 64, F16), (5e5, 128, BF16), (1e6, 128, F16)]):
        gen = torch.Generator(device="cuda").manual_seed(i)
        x = torch.randn(3, 40, 6, D, generator=gen, device="cuda").to(dtype)
        calls = [make(40, 4, 2, D, n=400, dtype=dtype, seed=i), make(3, 2, 2, D, n=70, new=True, dtype=dtype, seed=i),
                 make(150, 2, 4, D, P=1500, new=True, dtype=dtype, seed=i), make(60, 1, 4, D, P=3000, dtype=dtype, seed=i)]
        jobs.append((theta, x, calls))

    def once(job, stream):
        theta, x, calls = job
        outs = [torch.zeros_like(x)] + [torch.zeros_like(q) for q, _ in calls]
        stream.wait_stream(torch.cuda.default_stream())
        kvx.qk_norm_rope(x, None, outs[0], None, rope_theta=theta, stream=stream)
        for (q, rows), out in zip(calls, outs[1:]):
            kvx.attend(q, out, stream=stream, **rows)
        return outs
    streams = [torch.cuda.Stream() for _ in jobs]
    want = [once(job, s) for job, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    found, errors = [[] for _ in jobs], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(30):
                    found[i].append(once(jobs[i], streams[i]))
        except Exception as e:      # noqa: BLE001 -- shown by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for w, runs in zip(want, found):
        assert len(runs) == 30 and all(torch.equal(a, b) for run in runs for a, b in zip(w, run))


@pytest.mark.parametrize("B,S,G,H,D", [(64, 300, 2, 1, 128), (50, 401, 4, 4, 64), (17, 1000, 3, 2, 128)])
def test_norm_of_few_heads_of_many_sequences(kvx, B, S, G, H, D):
    """Several sequences' tokens of one position go to one warp here."""
    gen = torch.Generator(device="cuda").manual_seed(S)
    qkv = torch.randn(B, S, G + 2 * H, D, generator=gen, device="cuda", dtype=F16)
    w = torch.ones(D, device="cuda") + 0.1 * torch.randn(D, generator=gen, device="cuda")
    q, k = qkv[:, :, :G], qkv[:, :, G:G + H]
    q_out = torch.full_like(q, float("nan"))
    k_out = torch.full((B, H, S, D), float("nan"), dtype=F16, device="cuda").transpose(1, 2)
    kvx.qk_norm_rope(q, k, q_out, k_out, rope_theta=5e5, q_weight=w, k_weight=w, eps=1e-6, pos0=77)
    torch.cuda.synchronize()
    at = (torch.arange(S, device="cuda") + 77).expand(B, S)
    for name, x, o in (("q", q, q_out), ("k", k, k_out)):
        y, size = ref.qk(x, w, at, 5e5, 1e-6)
        ref.check(name, o, y, ref.qk_bound(y, size, F16))
