// AdamW over many tensors in one launch, optimizer states in 32 or in 8 bits (sm_100a).
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   p' = p - lr (m' c1 / (sqrt(v' c2) + eps) + wd p),   c1 = 1 / (1 - b1^t), c2 = 1 / (1 - b2^t)
//
// 8-bit states come in blocks of 256 elements that share one fp32 scale, the block's largest
// magnitude.  The codes are laid out by square roots, which is where the update needs them:
//   m = scale sign(q) (q / 127)^2   q in -127 .. 127      (block-relative steps of 1.6 % at the top)
//   v = scale (q / 255)^4           q in 0 .. 255         (sqrt(v), the divisor, by squares)
// v > 0 never rounds to 0: the update divides by its root, and a zero there with m left would
// be a step of m / eps.  Everything between decode and encode is fp32.
//
// Bound by HBM: p is read and written, g read, the states read and written: 28 B per element with
// fp32 throughout, 16 B with 8-bit states.  A warp works one block (8 elements a lane), so a scale
// is one warp reduction.
#include "common.cuh"
#include "internal.h"

#include <algorithm>
#include <cmath>

namespace soup {

namespace {

constexpr int BLOCK = ADAMW_BLOCK;
constexpr int LAUNCH_TENSORS = 640;  // descriptors of one launch: 32 KB of kernel parameters hold 800

struct AdamTensor {
  void* p;
  const void* g;
  uint16_t* pb;
  long long n;
  int aligned;  // p, g and pb on 16 bytes
};
struct Hyper {
  float lr, b1, b2, g1, g2, eps, wd, bc1, bc2;  // g = 1 - b
};
struct AdamArgs {
  void *m, *v;
  float *m_scale, *v_scale;
  const float* hp;
  Hyper k;
  int count;
  long long blocks;      // of this launch
  long long block0;      // state block of this launch's first
  long long first[LAUNCH_TENSORS];  // first block of each tensor, from this launch's first
  AdamTensor t[LAUNCH_TENSORS];
};

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(uint16_t* p, float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  *p = *reinterpret_cast<const uint16_t*>(&b);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_bf16x2(w[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ float m_value(int q, float scale) {
  const float r = static_cast<float>(q) * (1.f / 127.f);
  return r * fabsf(r) * scale;
}
__device__ __forceinline__ float v_value(int q, float scale) {
  const float r = static_cast<float>(q) * (1.f / 255.f), r2 = r * r;
  return r2 * r2 * scale;
}
// x / scale for 0 <= x <= scale, also where 1 / scale leaves fp32's range
struct Ratio {
  float up, inv;
  __device__ explicit Ratio(float scale) {
    up = scale < 1e-30f ? 18446744073709551616.f : 1.f;
    inv = scale > 0.f ? 1.f / (scale * up) : 0.f;
  }
  __device__ float operator()(float x) const { return x * up * inv; }
};
// The largest of 256 magnitudes of a warp: non-negative floats order like their bits, and so does a
// NaN above every number, which therefore reaches the scale instead of being lost in it.
__device__ __forceinline__ float block_top(const float (&x)[8]) {
  unsigned top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(fabsf(x[j])));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

template <typename P, typename G, bool BITS8>
__global__ void __launch_bounds__(256) adamw_multi_kernel(const __grid_constant__ AdamArgs a) {
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const long long w = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  // a run of blocks per warp
  const long long lo = a.blocks * w / warps, hi = a.blocks * (w + 1) / warps;
  if (lo >= hi) return;
  Hyper k = a.k;
  if (a.hp) {
    k.lr = a.hp[0];
    k.bc1 = a.hp[1];
    k.bc2 = a.hp[2];
  }
  int i = 0;  // the tensor of block lo
  for (int step = 512; step > 0; step >>= 1)
    if (i + step < a.count && a.first[i + step] <= lo) i += step;
  for (long long b = lo; b < hi; ++b) {
    while (i + 1 < a.count && a.first[i + 1] <= b) ++i;
    const AdamTensor& t = a.t[i];
    const long long e = (b - a.first[i]) * BLOCK + lane * 8;  // this lane's first element
    const int n = static_cast<int>(max(0ll, min(8ll, t.n - e)));
    const long long at = (a.block0 + b) * BLOCK + lane * 8;   // ... and its place in the states
    P* p = static_cast<P*>(t.p) + e;
    const G* g = static_cast<const G*>(t.g) + e;
    float pv[8], gv[8], m[8], v[8];
    const bool whole = n == 8 && t.aligned;
    if (whole) {
      load8(p, pv);
      load8(g, gv);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        pv[j] = j < n ? load_f(p + j) : 0.f;
        gv[j] = j < n ? load_f(g + j) : 0.f;
      }
    }
    if (BITS8) {
      const uint2 mq = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.m) + at);
      const uint2 vq = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + at);
      const float ms = a.m_scale[a.block0 + b], vs = a.v_scale[a.block0 + b];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t mw = (j < 4 ? mq.x : mq.y) >> (8 * (j & 3)), vw = (j < 4 ? vq.x : vq.y) >> (8 * (j & 3));
        m[j] = m_value(static_cast<int8_t>(mw & 255u), ms);
        v[j] = v_value(static_cast<int>(vw & 255u), vs);
      }
    } else {
      load8(static_cast<const float*>(a.m) + at, m);
      load8(static_cast<const float*>(a.v) + at, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = k.b1 * m[j] + k.g1 * gv[j];
      v[j] = k.b2 * v[j] + k.g2 * gv[j] * gv[j];
      const float mh = m[j] * k.bc1, vh = v[j] * k.bc2;
      pv[j] = pv[j] - k.lr * (mh / (sqrtf(vh) + k.eps) + k.wd * pv[j]);
    }
    if (BITS8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= n) m[j] = v[j] = 0.f;  // behind the tensor's end
      const float ms = block_top(m), vs = block_top(v);
      const Ratio mr(ms), vr(vs);
      uint32_t mq[2] = {0, 0}, vq[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = static_cast<int>(rintf(127.f * sqrtf(mr(fabsf(m[j])))));
        const int u = static_cast<int>(rintf(255.f * sqrtf(sqrtf(vr(v[j])))));
        mq[j >> 2] |= static_cast<uint32_t>((m[j] < 0.f ? -q : q) & 255) << (8 * (j & 3));
        vq[j >> 2] |= static_cast<uint32_t>(max(u, v[j] > 0.f ? 1 : 0)) << (8 * (j & 3));
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + at) = make_uint2(mq[0], mq[1]);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + at) = make_uint2(vq[0], vq[1]);
      if (lane == 0) {
        a.m_scale[a.block0 + b] = ms;
        a.v_scale[a.block0 + b] = vs;
      }
    } else if (n == 8) {
      store8(static_cast<float*>(a.m) + at, m);
      store8(static_cast<float*>(a.v) + at, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) {
          static_cast<float*>(a.m)[at + j] = m[j];
          static_cast<float*>(a.v)[at + j] = v[j];
        }
    }
    if (whole) {
      store8(p, pv);
      if (t.pb) store8(t.pb + e, pv);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) {
          store_f(p + j, pv[j]);
          if (t.pb) store_f(t.pb + e + j, pv[j]);
        }
    }
  }
}

// The values 8-bit states stand for, rounded once to bf16.
__global__ void adamw_values_kernel(const uint8_t* __restrict__ m, const uint8_t* __restrict__ v,
                                    const float* __restrict__ m_scale, const float* __restrict__ v_scale, long long blocks,
                                    uint16_t* __restrict__ mo, uint16_t* __restrict__ vo) {
  const long long b = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (b >= blocks) return;
  const long long at = b * BLOCK + (threadIdx.x & 31) * 8;
  const uint2 mq = *reinterpret_cast<const uint2*>(m + at), vq = *reinterpret_cast<const uint2*>(v + at);
  const float ms = m_scale[b], vs = v_scale[b];
  float mf[8], vf[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mf[j] = m_value(static_cast<int8_t>(((j < 4 ? mq.x : mq.y) >> (8 * (j & 3))) & 255u), ms);
    vf[j] = v_value(static_cast<int>(((j < 4 ? vq.x : vq.y) >> (8 * (j & 3))) & 255u), vs);
  }
  store8(mo + at, mf);
  store8(vo + at, vf);
}

template <typename P, typename G>
void launch(const AdamArgs& a, bool bits8, unsigned grid, cudaStream_t st) {
  if (bits8)
    adamw_multi_kernel<P, G, true><<<grid, 256, 0, st>>>(a);
  else
    adamw_multi_kernel<P, G, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t adamw_multi_launch(const soup_adamw_tensor* tensors, int count, const soup_adamw_options& o, void* m, void* v,
                               float* m_scale, float* v_scale, const float* hp, cudaStream_t st) {
  const bool p_bf16 = o.params_bf16 != 0, g_bf16 = o.grads_bf16 != 0;
  AdamArgs a;
  a.m = m;
  a.v = v;
  a.m_scale = m_scale;
  a.v_scale = v_scale;
  a.hp = hp;
  a.k.lr = static_cast<float>(o.lr);
  a.k.b1 = static_cast<float>(o.beta1);
  a.k.b2 = static_cast<float>(o.beta2);
  a.k.g1 = static_cast<float>(1.0 - o.beta1);
  a.k.g2 = static_cast<float>(1.0 - o.beta2);
  a.k.eps = static_cast<float>(o.eps);
  a.k.wd = static_cast<float>(o.weight_decay);
  a.k.bc1 = hp ? 1.f : static_cast<float>(1.0 / (1.0 - std::pow(o.beta1, o.step)));
  a.k.bc2 = hp ? 1.f : static_cast<float>(1.0 / (1.0 - std::pow(o.beta2, o.step)));
  long long block0 = 0;
  for (int i0 = 0; i0 < count; i0 += LAUNCH_TENSORS) {
    a.count = std::min(LAUNCH_TENSORS, count - i0);
    a.block0 = block0;
    a.blocks = 0;
    for (int i = 0; i < a.count; ++i) {
      const soup_adamw_tensor& t = tensors[i0 + i];
      const uintptr_t all = reinterpret_cast<uintptr_t>(t.p) | reinterpret_cast<uintptr_t>(t.g) |
                            reinterpret_cast<uintptr_t>(t.p_bf16_copy);
      a.t[i] = AdamTensor{t.p, t.g, t.p_bf16_copy, t.n, (all & 15u) == 0};
      a.first[i] = a.blocks;
      a.blocks += (t.n + BLOCK - 1) / BLOCK;
    }
    block0 += a.blocks;
    if (a.blocks == 0) continue;
    const long long want = (a.blocks + 7) / 8;
    const unsigned grid = static_cast<unsigned>(std::min<long long>(want, 8ll * device_sm_count()));
    if (p_bf16)
      g_bf16 ? launch<uint16_t, uint16_t>(a, m_scale != nullptr, grid, st) : launch<uint16_t, float>(a, m_scale != nullptr, grid, st);
    else
      g_bf16 ? launch<float, uint16_t>(a, m_scale != nullptr, grid, st) : launch<float, float>(a, m_scale != nullptr, grid, st);
    ++g_kernel_launches;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t adamw_values_launch(const uint8_t* m, const uint8_t* v, const float* m_scale, const float* v_scale, long long n,
                                uint16_t* mo, uint16_t* vo, cudaStream_t st) {
  const long long blocks = n / BLOCK;
  if (blocks <= 0) return cudaSuccess;
  adamw_values_kernel<<<static_cast<unsigned>((blocks + 7) / 8), 256, 0, st>>>(m, v, m_scale, v_scale, blocks, mo, vo);
  ++g_kernel_launches;
  return cudaGetLastError();
}

}  // namespace soup
