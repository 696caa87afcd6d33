"""The batch-invariant mode is process-wide and another thread may switch it at
any time, so a call reads it once: the mode whose workspace it checks is the mode
that it launches in.  Here the host layer (api.cu) is linked to stand-ins for the
kernels' launchers and to a mode that changes at every read; no device is needed."""
import os
import subprocess

from dsa_sparse_attention_index_gb300 import build

STANDINS = r"""
#include <cstdio>
#include "internal.h"
namespace dsa {
static int reads = 0, start = 0, checked = -1, launched = -1;
bool mla_batch_invariant_on() { return (start + reads++) & 1; }
static size_t size_of(bool inv) { checked = inv; return 1024; }
size_t dense_mla_workspace_bytes(int, int, bool inv) { return size_of(inv); }
dsa_status_t launch_dense_mla(const dsa_paged_cache_t&, const dsa_batch_t&, const uint16_t*, float, bool inv, uint16_t*,
                              float*, void*, int32_t*, cudaStream_t) { launched = inv; return DSA_OK; }
size_t mla_workspace_bytes(int, int, bool inv) { return size_of(inv); }
dsa_status_t launch_sparse_mla(const dsa_paged_cache_t&, const dsa_batch_t&, const uint16_t*, const int32_t*, int, float,
                               bool inv, uint16_t*, float*, void*, int32_t*, cudaStream_t, const int32_t*) {
  launched = inv;
  return DSA_OK;
}
size_t topk_workspace_bytes(int, int, int) { return 0; }
dsa_status_t launch_index_scores(const dsa_paged_cache_t&, const dsa_batch_t&, const uint8_t*, const float*, void*, bool,
                                 int64_t, int32_t*, cudaStream_t) { return DSA_OK; }
dsa_status_t launch_topk(const float*, int64_t, const int32_t*, const int32_t*, int, int, int, int, int32_t*, void*, int32_t*,
                         cudaStream_t, const TopkPhys&) { return DSA_OK; }
}  // namespace dsa
using namespace dsa;
int main() {
  void* at = reinterpret_cast<void*>(size_t(1) << 20);   // checked, never followed
  dsa_paged_cache_t c = {at, 45312, 0, 36864, 64, 10, DSA_KEY_FP8_E4M3, 1.0f, DSA_LATENT_FP8_E4M3};
  dsa_batch_t b = {static_cast<int32_t*>(at), static_cast<int32_t*>(at), 8, 2, 1, 500};
  uint16_t* u = static_cast<uint16_t*>(at);
  float* f = static_cast<float*>(at);
  int32_t* i = static_cast<int32_t*>(at);
  for (start = 0; start < 2; ++start) {
#define CALL(name, ...)                                                                       \
  reads = 0, checked = launched = -1;                                                         \
  if (name(__VA_ARGS__) != DSA_OK || launched < 0) return printf("%s not launched\n", #name), 1; \
  if (reads != 1 || checked != launched || launched != start)                                 \
    return printf("%s: %d reads, checked %d, launched %d\n", #name, reads, checked, launched), 1;
    CALL(dense_mla_decode, &c, &b, u, 1.0f, u, f, at, 1024, i, nullptr)
    CALL(sparse_mla_decode, &c, &b, u, i, 64, 1.0f, u, f, at, 1024, i, nullptr)
    CALL(dsa_decode_step, &c, &b, static_cast<uint8_t*>(at), f, u, 64, 1.0f, u, f, nullptr, 0, nullptr, nullptr, at, 1 << 20, i,
         nullptr)
  }
  return 0;
}
"""


def test_the_mode_is_read_once_per_call(tmp_path):
    src, exe = tmp_path / "standins.cu", tmp_path / "standins"
    src.write_text(STANDINS)
    include = os.path.join(os.path.dirname(build.HERE), "include")
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I", include,
                        os.path.join(build.CSRC, "api.cu"), str(src), "-o", str(exe),
                        "-Xlinker", "--unresolved-symbols=ignore-all"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
