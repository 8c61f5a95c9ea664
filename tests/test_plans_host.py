"""How paged attention and the scan cut their work (csrc/gdn_plan.h), compiled for the host under
sanitizers: over the sizes that a descriptor may have, every key and every chunk is in exactly one
part, and the kernels exist for what is chosen."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "gdn_plan.h"
using namespace gdn;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s; n %d total %lld heads %d on %d of %d, keys %d, bf16 %d: decode %d rows %d waves %d splits %d keys %d\n", \
    __LINE__, #x, n, (long long)total, h_q, h_kv, d, kv, bf16, p.decode, p.rows, p.waves, p.splits, p.split_keys); return 1; } } while (0)
static int attention(int64_t total, int n, int h_q, int h_kv, int d, int kv, int bf16)
{
    const AttnPlan p = attn_plan(total, n, h_q, h_kv, d, kv, bf16);
    CHECK(p.splits >= 1 && p.split_keys >= 1);
    CHECK(p.split_keys % (p.decode || !bf16 ? 32 : 64) == 0);
    CHECK((int64_t)p.splits * p.split_keys >= kv);
    CHECK(p.splits == 1 || (int64_t)(p.splits - 1) * p.split_keys < kv);
    CHECK((int64_t)(p.splits - 1) * p.split_keys + p.split_keys <= 0x7fffffff);      // the kernels' keys are 32-bit
    const int row = d * (bf16 ? 2 : 4), waves = decode_waves(row);
    if (p.decode) {
        CHECK(p.rows == 16 || (p.rows == 32 && bf16 && d != 128));
        CHECK(p.waves == waves || (decode_wide(row) && p.waves == 2 * waves));
    } else {
        CHECK(bf16 ? p.rows == 128 || p.rows == 256 : p.rows == 64);
    }
    // splits do not multiply workgroups that are many already
    if (p.decode && kv >= 4096) {
        const int64_t tiles = total * (h_q / h_kv) / p.rows, chains = (tiles > n ? tiles : n) * h_kv;
        CHECK(p.splits == 1 || p.splits * chains <= 2 * 8192 + chains);
    }
    return 0;
}
static int scan(int n, int h, int k, int v, int bf16, int64_t tokens)
{
    const int32_t s = scan_segments(n, h, k, v, bf16, tokens);
    const int64_t chunks = (tokens + kScanChunk - 1) / kScanChunk;
    if (s < 1 || s > (chunks > 1 ? chunks : 1)) {
        printf("scan: %d sequences, %d heads of %d x %d, %lld tokens: %d segments\n", n, h, k, v, (long long)tokens, s);
        return 1;
    }
    return 0;
}
int main()
{
    const int64_t seqs[] = {1, 2, 3, 17, 64, 300, 1023, 1024, 1025, 2048, 4095, 4096, 4097, 8192, 16384, 32768, 100000, 1 << 24, 0x7fffffff};
    const int keys[] = {0, 1, 31, 63, 64, 257, 4095, 4096, 4097, 32768, 100001, 1 << 20, 1 << 27, (1 << 27) + 1, 1 << 28, 1 << 29, (1 << 30) - 1, 1 << 30};
    const int64_t each[] = {0, 1, 2, 40, 1000};
    for (int64_t n : seqs) for (int kv : keys) for (int64_t e : each) for (int h_kv : {1, 2, 8, 32, 1 << 20}) for (int g : {1, 3, 8, 32}) for (int d : {64, 128, 256}) for (int bf16 : {0, 1}) {
        const int64_t total = n * e, h_q = (int64_t)h_kv * g;
        if (total > 0x7fffffff || total * h_q > 0x7fffffff || h_q * d > 0x7fffffff) continue;   // refused by the calls
        if (attention(total, (int)n, (int)h_q, h_kv, d, kv, bf16)) return 1;
    }
    for (int64_t n : seqs) for (int64_t t : {0LL, 1LL, 64LL, 65LL, 7001LL, 32768LL, 1000000LL, 0x7fffffffLL}) for (int h : {1, 4, 32, 1 << 20})
        for (int k : {64, 128}) for (int v : {64, 128}) for (int bf16 : {0, 1}) if (scan((int)n, h, k, v, bf16, t)) return 1;
    puts("plans: ok");
    return 0;
}
"""


@pytest.mark.parametrize("san", [None, "address,undefined"])
def test_plans_of_all_sizes(tmp_path, san):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "plans.cpp", str(tmp_path / "plans")
    src.write_text(PROGRAM)
    cmd = ["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "gated_deltanet_state_gdn_amd", "csrc"), str(src), "-o", exe]
    subprocess.check_call(cmd + (["-fsanitize=" + san, "-fno-sanitize-recover=all"] if san else []))
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "ok" in p.stdout, p.stdout + p.stderr[-2000:]


def test_workspaces_of_loose_bounds():
    """The largest bound on kv_len, by chains of keys around where splits end: the workspace is the
    status word, and neither the query nor a call divides by nothing."""
    import gated_deltanet_state_gdn_amd as gdn
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built here")
    for n, h_kv, kv in ((2048, 8, 1 << 30), (4096, 8, 1 << 30), (100000, 8, 1 << 30), (300, 32, 1 << 30), (32768, 8, 1 << 27)):
        d = gdn._lib.GdnPagedDesc(n_seqs=n, h_q=h_kv, h_kv=h_kv, d=64, dtype=1, page_size=16, n_pages=10, max_pages=1 << 26,
                                  max_kv_len=kv, scale=0.1, total_tokens=n, q_stride=h_kv * 64, o_stride=h_kv * 64,
                                  page_stride=1 << 15, token_stride=h_kv * 64, head_stride=64)
        assert gdn.gdn_paged_workspace_bytes(d) == 256
