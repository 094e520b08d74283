// Attention of one new token per sequence over a paged key-value cache:
//   s_t = scale * q . k_t,  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),
// one pass over the tokens with a running maximum m and sum l: when m grows,
// l and o so far are multiplied by exp(m_old - m_new).
#include <cfloat>
#include <cmath>

#include "attn_common.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Dec {
  const char *k, *v;                 // this layer's pools
  const int32_t *table, *lens, *seqs;
  int32_t* status;
  int num_pages, max_seqs, max_pages, page_shift, kv_heads, D;
  const void* q;
  void* out;
  float* lse;
  long long q_token, q_head, out_token, out_head;
  int n, heads, group, window;
  float scale;
};

// The plain kernel, for every type and head size: one block per (sequence, key
// head, GC query heads).  Eight lanes share a token (lane e of them holds the
// 16-byte chunks e, e + 8, ... of its key and value), so a warp works on four
// tokens; every lane group keeps its own running softmax and the block's groups
// are joined at the end through shared memory.
constexpr int kPlainWarps = 8;

template <typename T, int NC, int GC>
__global__ void __launch_bounds__(kPlainWarps * 32) k_decode_plain(const Dec a) {
  constexpr int W = 16 / sizeof(T);
  extern __shared__ float sm[];      // [groups of lanes][GC][D + 2]
  const int lane = threadIdx.x & 31, e = lane & 7;
  const int grp = threadIdx.x >> 3, groups = kPlainWarps * 4;
  const int chunks_of_heads = (a.group + GC - 1) / GC;
  const int i = blockIdx.y, kh = blockIdx.x / chunks_of_heads, g0 = blockIdx.x % chunks_of_heads * GC;
  const int row = a.seqs[i];
  const bool ok = (unsigned)row < (unsigned)a.max_seqs;
  int len = ok ? a.lens[row] : 0;
  const long long cap = (long long)a.max_pages << a.page_shift;
  if (!ok || len < 0 || len > cap) {
    if (threadIdx.x == 0) atomicCAS(a.status, MOE_KV_OK, MOE_KV_BAD_SEQ);
    len = 0;
  }
  const int from = a.window > 0 && len > a.window ? len - a.window : 0;
  const int D = a.D, units = D / W;
  float q[GC][NC][W], o[GC][NC][W], m[GC], l[GC];
#pragma unroll
  for (int g = 0; g < GC; ++g) {
    m[g] = -INFINITY, l[g] = 0.f;
    const int h = kh * a.group + (g0 + g < a.group ? g0 + g : a.group - 1);
    const T* qp = (const T*)a.q + i * a.q_token + h * a.q_head;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int d = (e + 8 * c) * W + w;
        q[g][c][w] = d < D ? Elem<T>::get(qp + d) * (a.scale * kLog2e) : 0.f;
        o[g][c][w] = 0.f;
      }
  }
  const long long head_elems = (long long)D << a.page_shift;
  const int pmask = (1 << a.page_shift) - 1;
  for (int t0 = from; t0 < len; t0 += groups) {      // uniform over the block
    const int t = t0 + grp;
    const bool live = t < len;
    int page = 0;
    if (live) {
      page = a.table[(size_t)row * a.max_pages + (t >> a.page_shift)];
      if ((unsigned)page >= (unsigned)a.num_pages) {
        if (e == 0) atomicCAS(a.status, MOE_KV_OK, MOE_KV_BAD_PAGE);
        page = -1;
      }
    }
    const bool use = live && page >= 0;
    const long long at = (((long long)page * a.kv_heads + kh) * head_elems) + (long long)(t & pmask) * D;
    float kk[NC][W];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int w = 0; w < W; ++w) kk[c][w] = 0.f;
      if (use && e + 8 * c < units) load_vec<T, W>((const T*)a.k + at + (e + 8 * c) * W, kk[c]);
    }
    float s[GC];
#pragma unroll
    for (int g = 0; g < GC; ++g) {
      s[g] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int w = 0; w < W; ++w) s[g] = fmaf(q[g][c][w], kk[c][w], s[g]);
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) s[g] += __shfl_xor_sync(kAll, s[g], x);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int w = 0; w < W; ++w) kk[c][w] = 0.f;
      if (use && e + 8 * c < units) load_vec<T, W>((const T*)a.v + at + (e + 8 * c) * W, kk[c]);
    }
    if (use) {
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        const float mn = fmaxf(m[g], s[g]);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[g] - base), p = exp2f(s[g] - base);
        m[g] = mn;
        l[g] = l[g] * f + p;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int w = 0; w < W; ++w) o[g][c][w] = fmaf(p, kk[c][w], o[g][c][w] * f);
      }
    }
  }
  // join the block's lane groups
  const int stride = D + 2;
#pragma unroll
  for (int g = 0; g < GC; ++g) {
    float* to = sm + (grp * GC + g) * stride;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int w = 0; w < W; ++w)
        if ((e + 8 * c) * W + w < D) to[(e + 8 * c) * W + w] = o[g][c][w];
    if (e == 0) to[D] = m[g], to[D + 1] = l[g];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < GC * D; x += blockDim.x) {
    const int g = x / D, d = x % D;
    if (g0 + g >= a.group) break;
    float mm = -INFINITY;
    for (int u = 0; u < groups; ++u) mm = fmaxf(mm, sm[(u * GC + g) * stride + D]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, oo = 0.f;
    for (int u = 0; u < groups; ++u) {
      const float* p = sm + (u * GC + g) * stride;
      const float f = exp2f(p[D] - base);
      ll = fmaf(p[D + 1], f, ll);
      oo = fmaf(p[d], f, oo);
    }
    const int h = kh * a.group + g0 + g;
    const bool some = !(ll == 0.f);
    Elem<T>::put((T*)a.out + i * a.out_token + h * a.out_head + d, some ? oo / ll : 0.f);
    if (d == 0 && a.lse) a.lse[(size_t)i * a.heads + h] = some ? base * kLn2 + logf(ll) : -INFINITY;
  }
}

template <typename T, int NC, int GC>
cudaError_t go_plain(const Dec& a, cudaStream_t s) {
  const size_t smem = (size_t)kPlainWarps * 4 * GC * (a.D + 2) * 4;
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(launch_state_mutex());
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (!set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(k_decode_plain<T, NC, GC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kPlainWarps * 4 * GC * (NC * 8 * (16 / (int)sizeof(T)) + 2) * 4);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  const dim3 grid((a.group + GC - 1) / GC * a.kv_heads, a.n);
  k_decode_plain<T, NC, GC><<<grid, kPlainWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t attn_decode_work_bytes(const moe_kv_pages& kv, int max_heads) { return 0; }

cudaError_t launch_attn_decode(const moe_kv_pages& kv, const DecodeArgs& m, cudaStream_t s) {
  if (m.n <= 0) return cudaSuccess;
  Dec a;
  const size_t e = kv.dtype == MOE_BF16 ? 2 : 4;
  const size_t layer = (size_t)kv.num_pages * kv.kv_heads * kv.page_tokens * kv.head_dim * e;
  a.k = (const char*)kv.k_d + m.layer * layer, a.v = (const char*)kv.v_d + m.layer * layer;
  a.table = kv.table_d, a.lens = kv.lens_d, a.seqs = m.seqs, a.status = kv.status_d;
  a.num_pages = kv.num_pages, a.max_seqs = kv.max_seqs, a.max_pages = kv.max_pages;
  a.page_shift = 0;
  while ((1 << a.page_shift) < kv.page_tokens) ++a.page_shift;
  a.kv_heads = kv.kv_heads, a.D = kv.head_dim;
  a.q = m.q, a.out = m.out, a.lse = m.lse;
  a.q_token = m.q_token, a.q_head = m.q_head, a.out_token = m.out_token, a.out_head = m.out_head;
  a.n = m.n, a.heads = m.heads, a.group = m.heads / kv.kv_heads, a.window = m.window, a.scale = m.scale;
  if (kv.dtype == MOE_BF16) {
    if (a.D <= 64) return go_plain<__nv_bfloat16, 1, 4>(a, s);
    if (a.D <= 128) return go_plain<__nv_bfloat16, 2, 4>(a, s);
    return go_plain<__nv_bfloat16, 4, 2>(a, s);
  }
  if (a.D <= 32) return go_plain<float, 1, 4>(a, s);
  if (a.D <= 64) return go_plain<float, 2, 4>(a, s);
  if (a.D <= 128) return go_plain<float, 4, 4>(a, s);
  return go_plain<float, 8, 2>(a, s);
}

}  // namespace moe
