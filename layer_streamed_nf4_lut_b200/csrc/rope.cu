// Rotary positions on their own (sm_100a): rotate-half or neighbouring pairs, all or the first part
// of each head, frequencies scaled for long contexts; forward and the rotation back.
//
//   angle(t, i) = position_t f_i;  (a, b) -> m (a cos - b sin, b cos + a sin);  the gradient of a
//   rotation is the rotation by -angle (times the same m).
//
// Bound by HBM: each value is read once and written once, 3 operations per value.  Angles of far
// positions need more than fp32 (position 10^6 at f = 1 is 1.6 10^5 turns): turns are formed and
// reduced in fp64, once per token and pair, and shared by the token's heads through shared memory.
#include "common.cuh"
#include "internal.h"

#include <algorithm>
#include <cmath>
#include <string>

namespace soup {

namespace {

struct RopeArgs {
  const void* x[2];  // q, k
  void* y[2];
  long long ldx[2], ldy[2];  // elements between tokens
  int heads[2];
  int head_dim, rotary;
  const int32_t* positions;
  float grow;
  int back;
  double turns[ROPE_MAX_PAIRS];  // f_i / 2 pi
};

// 8 values as fp32, whichever type they are stored in
template <typename E>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  __device__ static void load(const uint16_t* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16x2(w[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
  __device__ static void store(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  __device__ static float get(const uint16_t* p) { return bf16_to_f32(*p); }
  __device__ static void put(uint16_t* p, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t*>(&b);
  }
};
template <>
struct Vec8<float> {
  __device__ static void load(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ static void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ static float get(const float* p) { return *p; }
  __device__ static void put(float* p, float v) { *p = v; }
};

// One block per token.  VEC: groups of 8 values (the rotated part and, with rotate-half, its halves
// are whole groups and every address is aligned), else value by value.
template <typename E, bool PAIRED, bool VEC>
__global__ void rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float cs[ROPE_MAX_PAIRS], sn[ROPE_MAX_PAIRS];
  const long long t = blockIdx.x;
  const int half = a.rotary / 2;
  const double pos = static_cast<double>(a.positions[t]);
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double turns = pos * a.turns[i];
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    cs[i] = c * a.grow;
    sn[i] = (a.back ? -s : s) * a.grow;
  }
  __syncthreads();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (a.heads[which] == 0) continue;
    const E* x = static_cast<const E*>(a.x[which]) + t * a.ldx[which];
    E* y = static_cast<E*>(a.y[which]) + t * a.ldy[which];
    const bool copies = static_cast<const void*>(x) != static_cast<void*>(y);
    constexpr int W = VEC ? 8 : 1;
    // work items of a head: its pairs (W first members, or W / 2 neighbouring pairs), then its tail
    const int turn = PAIRED ? (VEC ? a.rotary / 8 : half) : half / W;
    const int per_head = turn + (copies ? (a.head_dim - a.rotary) / W : 0);
    for (int i = threadIdx.x; i < per_head * a.heads[which]; i += blockDim.x) {
      const int hd = i / per_head, k = i % per_head;
      const E* xh = x + hd * a.head_dim;
      E* yh = y + hd * a.head_dim;
      if (k >= turn) {
        const int c = a.rotary + (k - turn) * W;
        if (VEC) {
          float v[8];
          Vec8<E>::load(xh + c, v);
          Vec8<E>::store(yh + c, v);
        } else {
          yh[c] = xh[c];
        }
      } else if (VEC && PAIRED) {
        float v[8];
        Vec8<E>::load(xh + 8 * k, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = v[2 * j], q = v[2 * j + 1], c = cs[4 * k + j], s = sn[4 * k + j];
          v[2 * j] = p * c - q * s;
          v[2 * j + 1] = q * c + p * s;
        }
        Vec8<E>::store(yh + 8 * k, v);
      } else if (VEC) {
        float v[8], w[8];
        Vec8<E>::load(xh + 8 * k, v);
        Vec8<E>::load(xh + half + 8 * k, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = v[j], q = w[j], c = cs[8 * k + j], s = sn[8 * k + j];
          v[j] = p * c - q * s;
          w[j] = q * c + p * s;
        }
        Vec8<E>::store(yh + 8 * k, v);
        Vec8<E>::store(yh + half + 8 * k, w);
      } else {
        const int i0 = PAIRED ? 2 * k : k, i1 = PAIRED ? 2 * k + 1 : k + half;
        const float p = Vec8<E>::get(xh + i0), q = Vec8<E>::get(xh + i1);
        Vec8<E>::put(yh + i0, p * cs[k] - q * sn[k]);
        Vec8<E>::put(yh + i1, q * cs[k] + p * sn[k]);
      }
    }
  }
}

}  // namespace

bool rope_config_ok(const soup_rope_config& c, std::string& why) {
  if (c.rotary_dim < 2 || !(c.theta > 1.0) || c.scaling < SOUP_ROPE_NONE || c.scaling > SOUP_ROPE_YARN ||
      c.theta > 1e300) {
    why = "rope: rotary_dim >= 2, theta > 1 and a known scaling are needed";
    return false;
  }
  if (c.scaling != SOUP_ROPE_NONE && !(c.factor >= 1.0 && c.factor < 1e9)) {
    why = "rope: a scaling factor of at least 1 is needed";
    return false;
  }
  if (c.scaling >= SOUP_ROPE_BY_PARTS &&
      (c.original_len < 1 || !(c.low_freq_factor >= 0.0) || !(c.high_freq_factor > c.low_freq_factor) ||
       !(c.high_freq_factor < 1e9))) {
    why = "rope: original_len >= 1 and 0 <= low_freq_factor < high_freq_factor are needed";
    return false;
  }
  return true;
}

void rope_frequencies(const soup_rope_config& c, double* freq, double* grow) {
  const double d = c.rotary_dim, pi = 3.14159265358979323846;
  // with one pair only the exponent d / (d - 2) has no value; that pair's frequency is 1 whatever theta
  const double theta = c.scaling == SOUP_ROPE_NTK && d > 2 ? c.theta * std::pow(c.factor, d / (d - 2.0)) : c.theta;
  for (int i = 0; i < c.rotary_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / d);
    if (c.scaling == SOUP_ROPE_LINEAR) f /= c.factor;
    if (c.scaling == SOUP_ROPE_BY_PARTS || c.scaling == SOUP_ROPE_YARN) {
      const double r = c.original_len * f / (2.0 * pi);
      const double g =
          std::min(1.0, std::max(0.0, (r - c.low_freq_factor) / (c.high_freq_factor - c.low_freq_factor)));
      f = g * f + (1.0 - g) * (f / c.factor);
    }
    freq[i] = f;
  }
  *grow = c.scaling == SOUP_ROPE_YARN ? 1.0 + 0.1 * std::log(c.factor) : 1.0;
}

cudaError_t rope_launch(const RopeCall& c, cudaStream_t st) {
  if (c.T <= 0 || c.heads[0] + c.heads[1] == 0) return cudaSuccess;
  RopeArgs a{};
  bool vec = c.rotary % (c.interleaved ? 8 : 16) == 0 && c.head_dim % 8 == 0;
  const int size = c.f32 ? 4 : 2;
  for (int w = 0; w < 2; ++w) {
    a.x[w] = c.x[w];
    a.y[w] = c.y[w];
    a.ldx[w] = c.ldx[w];
    a.ldy[w] = c.ldy[w];
    a.heads[w] = c.heads[w];
    if (c.heads[w] && (((reinterpret_cast<uintptr_t>(c.x[w]) | reinterpret_cast<uintptr_t>(c.y[w])) & 15u) ||
                       (c.ldx[w] * size) % 16 || (c.ldy[w] * size) % 16))
      vec = false;
  }
  a.head_dim = c.head_dim;
  a.rotary = c.rotary;
  a.positions = c.positions;
  a.grow = c.grow;
  a.back = c.back;
  for (int i = 0; i < c.rotary / 2; ++i) a.turns[i] = c.freq[i] / 6.283185307179586476925;
  const int items = (c.heads[0] + c.heads[1]) * c.head_dim / (vec ? 16 : 2);
  const int threads = std::max(64, std::min(256, (items + 31) / 32 * 32));
  const dim3 grid(static_cast<unsigned>(c.T));
#define SOUP_ROPE(E)                                                                          \
  do {                                                                                        \
    if (c.interleaved)                                                                        \
      vec ? rope_kernel<E, true, true><<<grid, threads, 0, st>>>(a)                           \
          : rope_kernel<E, true, false><<<grid, threads, 0, st>>>(a);                         \
    else                                                                                      \
      vec ? rope_kernel<E, false, true><<<grid, threads, 0, st>>>(a)                          \
          : rope_kernel<E, false, false><<<grid, threads, 0, st>>>(a);                        \
  } while (0)
  if (c.f32)
    SOUP_ROPE(float);
  else
    SOUP_ROPE(uint16_t);
#undef SOUP_ROPE
  ++g_kernel_launches;
  return cudaGetLastError();
}

}  // namespace soup
