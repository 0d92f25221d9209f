"""Child process of test_attention_wait_timeout.

With PCD_WAIT_LIMIT_MS set far below a copy's latency (read at the process's
first call), the pipeline waits of the attention for many rows give up wherever
one outlasts a hardware try-wait window.  The kernel then records an error,
drains its copies and MMAs and returns; every row it did not finish is NaN, with
its log-sum-exp, and all others are right, whichever waits ran out.  Calls
without such waits work in the same process afterwards.  Prints the errors seen;
exits 0 only if every call went as stated.
"""
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import paged_ref as R  # noqa: E402
from test_gpu_paged import attend_case  # noqa: E402


def main():
    from constrained_decoding_gb300 import paged
    assert float(os.environ["PCD_WAIT_LIMIT_MS"]) < 1e-3
    seen = []
    for dim in (64, 128):
        for dtype in ("f16", "bf16"):
            for q_lens, hint in (([300, 40], 1), ([300, 40], 20000), ([18, 10], 1), ([18, 10], 20000)):
                a = attend_case("e4m3", dtype, 16, dim, 7, 1, q_lens, [2000, 1500], 3, "slot")
                want, wl, ob, lb = R.attention(*a, True, dim ** -0.5)
                odd = torch.empty(a[0].numel() + 1, dtype=a[0].dtype, device="cuda")[1:].view(a[0].shape)
                odd.copy_(a[0])
                for q in (a[0], odd):
                    err = torch.zeros(1, dtype=torch.int32, device="cuda")
                    out, lse = paged.pcd_k_paged_attention(q, *a[1:], max_kv=hint, return_lse=True, err=err)
                    failed = torch.isnan(lse)
                    assert torch.equal(torch.isnan(out).any(-1), failed) and torch.equal(torch.isnan(out).all(-1), failed)
                    assert torch.all(((out.double() - want).abs() <= ob) | failed[..., None])
                    assert torch.all(((lse.double() - wl).abs() <= lb) | failed)
                    assert int(err) in (1, 2, 3) if failed.any() else int(err) in (0, 1, 2, 3)
                    seen.append((int(err), int(failed.sum())))
    print("errors and failed rows", seen, flush=True)
    a = attend_case("e4m3", "f16", 16, 128, 7, 1, [1, 1], [2000, 1500], 3)
    want, _, ob, _ = R.attention(*a, True, 128 ** -0.5)
    assert torch.all((paged.pcd_k_paged_attention(*a).double() - want).abs() <= ob)
    print("other calls ok", flush=True)


if __name__ == "__main__":
    main()
