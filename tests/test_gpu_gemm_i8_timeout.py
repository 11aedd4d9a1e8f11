"""The int8 product's bounded waits, made to run out on purpose (no fault:
every wait gives up at its deadline, records DFLASH_ERR_TIMEOUT, drains what it
has in flight and returns), on its four paths: weight streaming, 2-CTA pairs,
single CTAs at the same sizes, and K split over clusters.  A child process
sets DFLASH_TIMEOUT_NS, read at every call, far below the call's time, then
clears it: the next call of the same process must be right.  The budget is each
wait's own.  The first is far below the time of a tile, for which the epilogue
waits, so its call must time out; the second is near it, so its call may also
complete."""
import json
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

pytestmark = pytest.mark.gpu

# a long K: the epilogue waits about 100 us for a tile's accumulator
CASES = [(8, 20000, 32768, {}, (2_000, 60_000)),
         (448, 20000, 32768, {}, (2_000, 60_000)),
         (448, 20000, 32768, {"DFLASH_PAIR": "0"}, (2_000, 60_000)),
         (8, 1000, 131056, {}, (2_000, 30_000))]


def child(case):
    sys.path[:0] = [ROOT, HERE]
    import torch
    import block_draft_selection_b200 as bds

    M, N, K, env, budgets = CASES[case]
    os.environ.update(env)
    g = torch.Generator(device="cuda").manual_seed(case)
    A = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    want = (A.double() @ B.double().t()).float() * sa[:, None] * sb[None]

    def call():
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        C = bds.dflash_gemm_i8(A, sa, B, sb, dev_status=status)
        torch.cuda.synchronize()
        return int(status), C

    codes, right = [], []
    call()
    for budget in budgets:
        os.environ["DFLASH_TIMEOUT_NS"] = str(budget)
        codes.append(call()[0])
        del os.environ["DFLASH_TIMEOUT_NS"]
        code, C = call()
        codes.append(code)
        right.append(bool(torch.equal(C, want)))
    print(json.dumps({"codes": codes, "right": right, "timeout_code": bds.DFLASH_ERR_TIMEOUT}), flush=True)


@pytest.mark.parametrize("case", range(len(CASES)), ids=["stream", "pairs", "single-ctas", "split"])
def test_wait_budget_runs_out_and_context_survives(case):
    out = subprocess.run([sys.executable, os.path.abspath(__file__), "--child", str(case)], cwd=ROOT,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-3000:]
    d = json.loads([l for l in out.stdout.splitlines() if l.startswith("{")][-1])
    T = d["timeout_code"]
    assert d["codes"][0] == T and d["codes"][1] == d["codes"][3] == 0 and d["codes"][2] in (0, T), d["codes"]
    assert all(d["right"])


if __name__ == "__main__" and "--child" in sys.argv:
    child(int(sys.argv[sys.argv.index("--child") + 1]))
