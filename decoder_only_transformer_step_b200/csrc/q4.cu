// Linear layers with 4-bit weights for decoding: quantisation of a weight
// matrix into signed 4-bit numbers with one scale per group of consecutive
// inputs, and the matrix-vector products of up to 16 rows that read it.
//
//   s[n, j] = bf16(max over group j of |w[n, k]| / 7)
//   q[n, k] = clamp(rint(w[n, k] / s[n, j]), -7, 7)   (0 where s is 0)
//   y[r, n] = sum_j s[n, j] sum_{k in group j} q[n, k] x[r, k]
//
// Storage: nibbles q + 8, byte j of a row holding k = 2j (low half) and
// 2j + 1; scales group-major [K / group][pitch], pitch = N rounded up to 8, so
// that the scales of a tile of output columns are consecutive.
#include "common.cuh"
#include "internal.h"

namespace {

// ------------------------------------------------------------- quantising --
// A block takes 32 rows x 256 inputs: a lane holds 8 consecutive inputs of
// each of the 4 rows of its warp (all loads in flight together), a group is
// 4, 8 or 16 neighbouring lanes.  The scales of the tile meet in shared memory
// and leave as runs of 32 columns.  Bound by HBM: 2 or 4 bytes a weight in,
// half a byte out.
constexpr int QZ_ROWS = 32, QZ_K = 256;

// rint(w / s), the division as IEEE rounds it: the product with the reciprocal
// r = 1 / s is within 7 * 2^-22 < 1e-5 of the quotient, so that the integers
// can differ only within that of a half; only there is the division made.
DEVI int q4_round(float w, float s, float r) {
  const float t = w * r;
  float q = rintf(t);
  if (!(fabsf(t - q) < 0.49999f)) q = rintf(w / s);
  return __float2int_rn(fminf(fmaxf(q, -7.f), 7.f));
}

template <typename T, int G>
__global__ void __launch_bounds__(256)
    q4_quantize_kernel(const T* w, long ldw, int N, int K, uint8_t* __restrict__ packed, bf16* __restrict__ scales,
                       long pitch) {
  constexpr int LG = G / 8;  // lanes of a group
  __shared__ bf16 sm[QZ_K / G][QZ_ROWS];
  pdl_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * QZ_ROWS, k0 = blockIdx.y * QZ_K, k = k0 + lane * 8;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + warp * 4 + i;
    if (n < N && k < K) {
      const T* p = w + (size_t)n * ldw + k;
      if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        v[i][0] = bf16lo(u.x); v[i][1] = bf16hi(u.x); v[i][2] = bf16lo(u.y); v[i][3] = bf16hi(u.y);
        v[i][4] = bf16lo(u.z); v[i][5] = bf16hi(u.z); v[i][6] = bf16lo(u.w); v[i][7] = bf16hi(u.w);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
        v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the largest magnitude as an unsigned integer: NaN above infinity above
    // every finite value, so that a group holding either gets such a scale
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7fffffffu);
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bf16 sb = __float2bfloat16_rn(__uint_as_float(top) / 7.f);
    const float s = __bfloat162float(sb), r = 1.f / s;
    const int n = n0 + warp * 4 + i;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) word |= (uint32_t)((s == 0.f ? 0 : q4_round(v[i][e], s, r)) + 8) << (4 * e);
    if (n < N && k < K) *reinterpret_cast<uint32_t*>(packed + ((size_t)n * K + k) / 2) = word;
    if (lane % LG == 0) sm[lane / LG][warp * 4 + i] = sb;
  }
  __syncthreads();
  // the columns between N and the pitch of the last row block get zero scales
  for (int i = threadIdx.x; i < QZ_K / G * QZ_ROWS; i += 256) {
    const int j = i / QZ_ROWS, c = i % QZ_ROWS;
    if (k0 + j * G < K && n0 + c < pitch) scales[(size_t)(k0 / G + j) * pitch + n0 + c] = sm[j][c];
  }
}

// The values the nibbles stand for, s q (exact in fp32, rounded once to bf16
// where T is bf16); one thread per 8 of them, 16 rows of a block sharing the
// sectors of the scales.
template <typename T>
__global__ void __launch_bounds__(256)
    q4_dequantize_kernel(const uint8_t* packed, const bf16* scales, long pitch, int group_shift, int N, int K,
                         T* __restrict__ out, long ldo) {
  pdl_start();
  const int k = (blockIdx.y * 32 + (threadIdx.x & 31)) * 8;
  if (k >= K) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = blockIdx.x * 16 + (threadIdx.x >> 5) + 8 * i;
    if (n >= N) continue;
    const uint32_t u = *reinterpret_cast<const uint32_t*>(packed + ((size_t)n * K + k) / 2);
    const float s = to_f(scales[(size_t)(k >> group_shift) * pitch + n]);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s * (float)((int)((u >> (4 * e)) & 15u) - 8);
    T* p = out + (size_t)n * ldo + k;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

// ------------------------------------------------- matrix-vector products --
// Bound by HBM reads of the nibbles.  The products run on mma.sync m16n8k16
// with the weights as A (16 output columns a warp tile) and the rows of x as
// B: at 13e12 weights/s (the copy bandwidth) CUDA-core multiply-adds of even
// one row would take more issue slots than there are, while a nibble reaches
// the tensor core in 1.4 instructions: bf16 bits 0x4300 | nibble are
// 128 + nibble, and one packed subtraction of 136 leaves q exactly.  The
// products of a group are summed in fp32 by the tensor core, with exact
// operands, and the group's sum is multiplied by its scale in fp32, so that
// no weight is rounded again.
//
// A block is 16 warps.  KS of them share a tile of 16 columns, each taking
// every KS-th stage of 128 inputs of the tile; their sums meet in shared memory in a
// fixed order.  Each warp copies its own stages (16 rows x 64 bytes and their
// scales) into a ring of its own with cp.async, several ahead, across tile
// borders: no block-wide wait stands in the stream.  The rows of x lie in
// shared memory as bf16 in the order in which the nibbles of a word unpack
// (0 4 1 5 2 6 3 7), so that a fragment is one 16-byte load.  Inputs too long
// for shared memory are split over the blocks of a cluster (up to 8), whose
// sums meet through distributed shared memory, again in a fixed order.
constexpr int Q4_WARPS = 16;
constexpr int Q4_COLS = 16;                    // output columns of a tile (the mma M)
constexpr int Q4_STAGE = 128;                  // inputs of a stage
constexpr int Q4_ROWPITCH = Q4_STAGE / 2 + 16; // bytes of a staged row: 8 rows' words then lie in 32 banks
constexpr int Q4_MAX_RING = 6;
constexpr int Q4_MAX_SPLIT = 8;
constexpr int Q4_PART_TILES = 16;              // tiles whose sums a cluster exchanges at once
constexpr int Q4_MAX_K = 32768;                // widest input
constexpr int Q4_SMEM = 227 * 1024;

struct Q4Args {
  const void* in;  // [rows, ldi]: bf16, or fp32 where in_f32 or ln
  long ldi;
  int in_f32, ln;  // ln: LayerNorm (eps 1e-5, biased variance) in front
  const bf16* ln_g;
  const bf16* ln_b;
  const uint8_t* W;  // [N, K / 2]
  const bf16* sc;    // [K / group, pitch]
  long pitch;
  const bf16* bias;  // [N] or NULL
  void* out;         // [rows, ldo]
  long ldo;
  int epi;           // Q4Epi
  int rows, N, K;
  int ks, split, kr, ring, w_early;
  void* kc;
  void* vc;
  const int32_t* pos;
  int d, H, hd, max_len;
};
enum Q4Epi : int { Q4_BF16 = 0, Q4_F32, Q4_QKV, Q4_RESID, Q4_GELU };

template <int G> constexpr int q4_slot() { return Q4_COLS * Q4_ROWPITCH + Q4_STAGE / G * Q4_COLS * 2; }
// elements of a staged row of x: an odd multiple of 64 bytes
inline int q4_xpitch(int kr) { return kr % 64 ? kr : kr + 32; }

DEVI void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
DEVI void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
DEVI void cp_wait(int pending) {  // at most `pending` of the newest groups still in flight
  switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
  }
}
DEVI uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
DEVI float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return __uint_as_float((uint32_t)v << 16);
}
DEVI uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
DEVI float4 ld_dsmem4(uint32_t addr, int rank) {
  const uint32_t a = mapa_shared(addr, rank);
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// nibbles i and i + 4 of w as bf16 q
DEVI uint32_t q4_pair(uint32_t w, int i) {
  const uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const uint32_t c = 0x43084308u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}
DEVI void q4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// eight fp32 / bf16 inputs, rounded to bf16, in the nibbles' order
DEVI uint4 q4_order(const float4& a, const float4& b) {
  return make_uint4(pack_bf16x2(a.x, b.x), pack_bf16x2(a.y, b.y), pack_bf16x2(a.z, b.z), pack_bf16x2(a.w, b.w));
}
DEVI uint4 q4_order(const uint4& u) {
  return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                    __byte_perm(u.y, u.w, 0x7632));
}
DEVI float4 q4_ld4(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}

// Inputs [k0, k0 + kn) of the rows -> xs [NR][xp] (rows past a.rows zero).
template <int NR>
DEVI void q4_stage_x(const Q4Args& a, bf16* xs, int xp, int k0, int kn, int warp, int lane) {
  if (a.ln) {
    // one warp a row, the row held in registers for its two statistics
    // (K <= 2048; the LayerNorm'd inputs are never split: k0 = 0, kn = K)
    constexpr int U = 8;
    const int K8 = a.K / 8;
    for (int r = warp; r < NR; r += Q4_WARPS) {
      bf16* dst = xs + (size_t)r * xp;
      if (r >= a.rows) {
        for (int i = lane; i < K8; i += 32) *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      const float* src = reinterpret_cast<const float*>(a.in) + (size_t)r * a.ldi;
      float4 v[U][2];
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = lane + 32 * u;
        v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < K8) {
          v[u][0] = *reinterpret_cast<const float4*>(src + 8 * i);
          v[u][1] = *reinterpret_cast<const float4*>(src + 8 * i + 4);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        s += ((v[u][0].x + v[u][0].y) + (v[u][0].z + v[u][0].w)) + ((v[u][1].x + v[u][1].y) + (v[u][1].z + v[u][1].w));
      const float mu = warp_sum(s) / a.K;
      float q = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (lane + 32 * u < K8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float t0 = v[u][h].x - mu, t1 = v[u][h].y - mu, t2 = v[u][h].z - mu, t3 = v[u][h].w - mu;
            q += (t0 * t0 + t1 * t1) + (t2 * t2 + t3 * t3);
          }
        }
      }
      const float rs = rsqrtf(warp_sum(q) / a.K + 1e-5f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = lane + 32 * u;
        if (i < K8) {
          float4 o[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 gg = q4_ld4(a.ln_g + 8 * i + 4 * h), bb = q4_ld4(a.ln_b + 8 * i + 4 * h);
            o[h] = make_float4((v[u][h].x - mu) * rs * gg.x + bb.x, (v[u][h].y - mu) * rs * gg.y + bb.y,
                               (v[u][h].z - mu) * rs * gg.z + bb.z, (v[u][h].w - mu) * rs * gg.w + bb.w);
          }
          *reinterpret_cast<uint4*>(dst + 8 * i) = q4_order(o[0], o[1]);
        }
      }
    }
    return;
  }
  constexpr int U = 8;  // loads in flight per thread
  const int n8 = kn / 8, total = NR * n8, nthr = Q4_WARPS * 32;
  for (int i0 = threadIdx.x; i0 < total; i0 += U * nthr) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * nthr, r = i / n8, c = i - r * n8;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < total && r < a.rows) {
        if (a.in_f32) {
          const float* p = reinterpret_cast<const float*>(a.in) + (size_t)r * a.ldi + k0 + 8 * c;
          v[u] = q4_order(*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4));
        } else {
          v[u] = q4_order(*reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.in) + (size_t)r * a.ldi + k0 +
                                                          8 * c));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * nthr, r = i / n8, c = i - r * n8;
      if (i < total) *reinterpret_cast<uint4*>(xs + (size_t)r * xp + 8 * c) = v[u];
    }
  }
}

// The epilogue of one lane's four sums of an n-tile: columns n0 + g,
// n0 + g + 8 (values 0 1, 2 3), rows r0 and r0 + 1 (values 0 2, 1 3).
DEVI void q4_epilogue(const Q4Args& a, const float4& s, int n0, int g, int r0) {
  const float v4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + g + 8 * (i >> 1), r = r0 + (i & 1);
    if (n >= a.N || r >= a.rows) continue;
    const float v = v4[i] + (a.bias ? to_f(a.bias[n]) : 0.f);
    const size_t at = (size_t)r * a.ldo + n;
    float* of = reinterpret_cast<float*>(a.out);
    bf16* ob = reinterpret_cast<bf16*>(a.out);
    switch (a.epi) {
      case Q4_BF16: ob[at] = from_f<bf16>(v); break;
      case Q4_F32: of[at] = v; break;
      case Q4_RESID: of[at] += v; break;
      case Q4_GELU: ob[at] = from_f<bf16>(gelu_f<false>(v)); break;
      default: {  // Q4_QKV: q to out, k and v into the cache at pos[r]
        if (n < a.d) {
          of[at] = v;
        } else {
          const int kind = n >= 2 * a.d, nn = n - a.d - kind * a.d, p = a.pos[r];
          if (p >= 0 && p < a.max_len) {
            bf16* plane = reinterpret_cast<bf16*>(kind ? a.vc : a.kc);
            plane[(((size_t)r * a.H + nn / a.hd) * a.max_len + p) * a.hd + nn % a.hd] = from_f<bf16>(v);
          }
        }
      }
    }
  }
}

template <int NT, int G>
__global__ void __launch_bounds__(Q4_WARPS * 32, 1) q4_gemv_kernel(const __grid_constant__ Q4Args a) {
  extern __shared__ __align__(128) uint8_t q4_smem[];
  constexpr int NR = 8 * NT;            // rows of x held
  constexpr int SLOT = q4_slot<G>();
  constexpr int GS = Q4_STAGE / G;      // groups of a stage
  constexpr int CG = G / 32;            // 32-input chunks of a group
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = a.split > 1 ? (int)cluster_ctarank() : 0;
  const int bx = blockIdx.x / a.split, gx = gridDim.x / a.split;
  const int k0 = rank * a.kr, kn = max(0, min(a.kr, a.K - k0));
  const int xp = a.kr % 64 ? a.kr : a.kr + 32;
  bf16* xs = reinterpret_cast<bf16*>(q4_smem);
  float4* red = reinterpret_cast<float4*>(q4_smem + (size_t)NR * xp * 2);       // [2][warps][NT][32]
  float4* part = red + 2 * Q4_WARPS * NT * 32;                                  // (split) [tiles][NT][32]
  uint8_t* ring0 = reinterpret_cast<uint8_t*>(part + (a.split > 1 ? Q4_PART_TILES * NT * 32 : 0));
  const uint32_t ring = smem_u32(ring0) + warp * a.ring * SLOT;
  const int ks = a.ks, grp = warp / ks, si = warp % ks, gpb = Q4_WARPS / ks;
  const int ntiles = (a.N + Q4_COLS - 1) / Q4_COLS, nst = (kn + Q4_STAGE - 1) / Q4_STAGE;
  const int tstep = gx * gpb;

  // the producer side of this warp's ring
  int pt = si < nst ? bx * gpb + grp : ntiles, ps = si, pslot = 0;
  auto issue = [&]() {
    if (pt < ntiles) {
      const uint32_t dst = ring + pslot * SLOT;
      const int kk = k0 + ps * Q4_STAGE, nseg = min(Q4_STAGE, k0 + kn - kk) / 32;
      const int n0 = pt * Q4_COLS;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = (lane >> 2) + 8 * h;
        const int n = min(n0 + row, a.N - 1);  // columns past N read the last one and are dropped
        if (t < nseg) cp_async16(dst + row * Q4_ROWPITCH + 16 * t, a.W + ((size_t)n * a.K + kk) / 2 + 16 * t);
      }
      // 16 columns of scales a group, 8 a copy (the pitch is a multiple of 8)
      if (lane < 2 * GS) {
        const int j = lane >> 1, c = n0 + 8 * (lane & 1);
        if (kk + j * G < k0 + kn && c < a.pitch)
          cp_async16(dst + Q4_COLS * Q4_ROWPITCH + lane * 16, a.sc + (size_t)(kk / G + j) * a.pitch + c);
      }
      ps += ks;
      if (ps >= nst) {
        ps = si;
        pt += tstep;
      }
    }
    cp_commit();
    pslot = pslot + 1 == a.ring ? 0 : pslot + 1;
  };

  pdl_trigger();
  // In the decode step no kernel writes weights and its first kernel lets its
  // successors start only after every kernel before the step has finished:
  // there (w_early) the first stages are requested before the wait.
  if (!a.w_early) pdl_wait();
  for (int i = 0; i < a.ring - 1; ++i) issue();
  if (a.w_early) pdl_wait();
  q4_stage_x<NR>(a, xs, xp, k0, kn, warp, lane);
  __syncthreads();

  const uint32_t xb = smem_u32(xs) + (uint32_t)(g * xp * 2 + 16 * t);
  int cslot = 0, par = 0, it = 0;
  const int ptg = Q4_PART_TILES / gpb;  // (split) tile passes between exchanges
  for (int base = bx * gpb; base < ntiles; base += tstep) {
    const int tile = base + grp;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    if (tile < ntiles) {
      for (int s = si; s < nst; s += ks) {
        cp_wait(a.ring - 2);
        __syncwarp();  // every lane's copies of this stage have landed; the slot before it is free
        issue();
        const uint32_t w = ring + cslot * SLOT + g * Q4_ROWPITCH + 4 * t;
        const uint32_t sc = ring + cslot * SLOT + Q4_COLS * Q4_ROWPITCH + 2 * g;
        const int nch = min(Q4_STAGE, kn - s * Q4_STAGE) / 32;
        const uint32_t xk = xb + s * Q4_STAGE * 2;
#pragma unroll
        for (int j = 0; j < GS; ++j) {
          if (j * CG < nch) {
            float c0[NT][4], c1[NT][4];
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) c0[m][i] = c1[m][i] = 0.f;
#pragma unroll
            for (int ch = j * CG; ch < (j + 1) * CG; ++ch) {
              const uint32_t wa = lds32(w + 16 * ch), wb = lds32(w + 8 * Q4_ROWPITCH + 16 * ch);
              const uint32_t p0 = q4_pair(wa, 0), p1 = q4_pair(wb, 0), p2 = q4_pair(wa, 1), p3 = q4_pair(wb, 1);
              const uint32_t p4 = q4_pair(wa, 2), p5 = q4_pair(wb, 2), p6 = q4_pair(wa, 3), p7 = q4_pair(wb, 3);
#pragma unroll
              for (int m = 0; m < NT; ++m) {
                const uint4 xv = lds128(xk + (uint32_t)(m * 8 * xp * 2) + 64 * ch);
                q4_mma(c0[m], p0, p1, p2, p3, xv.x, xv.y);
                q4_mma(c1[m], p4, p5, p6, p7, xv.z, xv.w);
              }
            }
            const float s0 = lds_bf16(sc + 32 * j), s1 = lds_bf16(sc + 32 * j + 16);
#pragma unroll
            for (int m = 0; m < NT; ++m) {
              acc[m][0] = fmaf(s0, c0[m][0] + c1[m][0], acc[m][0]);
              acc[m][1] = fmaf(s0, c0[m][1] + c1[m][1], acc[m][1]);
              acc[m][2] = fmaf(s1, c0[m][2] + c1[m][2], acc[m][2]);
              acc[m][3] = fmaf(s1, c0[m][3] + c1[m][3], acc[m][3]);
            }
          }
        }
        cslot = cslot + 1 == a.ring ? 0 : cslot + 1;
      }
    }
    float4 tot[NT];
#pragma unroll
    for (int m = 0; m < NT; ++m) tot[m] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
    if (ks > 1) {
      // two buffers in turn: a buffer is written again only after the next
      // barrier, which the warp that read it has then reached
      float4* rb = red + par * (Q4_WARPS * NT * 32);
      par ^= 1;
#pragma unroll
      for (int m = 0; m < NT; ++m) rb[(warp * NT + m) * 32 + lane] = tot[m];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(ks * 32) : "memory");
      if (si == 0) {
        for (int x = 1; x < ks; ++x) {
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            const float4 q = rb[((warp + x) * NT + m) * 32 + lane];
            tot[m].x += q.x;
            tot[m].y += q.y;
            tot[m].z += q.z;
            tot[m].w += q.w;
          }
        }
      }
    }
    if (a.split == 1) {
      if (si == 0 && tile < ntiles)
#pragma unroll
        for (int m = 0; m < NT; ++m) q4_epilogue(a, tot[m], tile * Q4_COLS, g, 8 * m + 2 * t);
    } else {
      // tiles of this block since the last exchange: slot (pass, group)
      const int pass = it % ptg;
      if (si == 0)
#pragma unroll
        for (int m = 0; m < NT; ++m) part[((pass * gpb + grp) * NT + m) * 32 + lane] = tot[m];
      const bool last = base + tstep >= ntiles;
      if (pass == ptg - 1 || last) {
        cluster_sync_all();
        // slot x is finished by rank x % split, one warp a slot
        const int pbase = base - pass * tstep, nslots = (pass + 1) * gpb;
        for (int x = rank + warp * a.split; x < nslots; x += Q4_WARPS * a.split) {
          const int tl = pbase + (x / gpb) * tstep + x % gpb;
          if (tl < ntiles) {
#pragma unroll
            for (int m = 0; m < NT; ++m) {
              const uint32_t at = smem_u32(part + (x * NT + m) * 32 + lane);
              float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
              for (int rk = 0; rk < a.split; ++rk) {
                const float4 q = ld_dsmem4(at, rk);
                sum.x += q.x;
                sum.y += q.y;
                sum.z += q.z;
                sum.w += q.w;
              }
              q4_epilogue(a, sum, tl * Q4_COLS, g, 8 * m + 2 * t);
            }
          }
        }
        cluster_sync_all();  // the slots are free again, and no block leaves while another reads it
      }
      ++it;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// How a product is spread over the machine: the k range of a block (the
// cluster split), the warps that share a tile and the depth of the rings.
struct Q4Plan {
  int split, kr, ks, ring, grid;
  size_t smem;
};
bool q4_plan(int rows, int N, int K, int group, bool ln, Q4Plan* p) {
  const int NR = rows <= 8 ? 8 : 16, NT = NR / 8;
  const int slot = Q4_COLS * Q4_ROWPITCH + Q4_STAGE / group * Q4_COLS * 2;
  const int nst = (K + Q4_STAGE - 1) / Q4_STAGE, ntiles = (N + Q4_COLS - 1) / Q4_COLS;
  for (p->split = 1; p->split <= Q4_MAX_SPLIT; p->split *= 2) {
    p->kr = p->split == 1 ? K : (nst + p->split - 1) / p->split * Q4_STAGE;
    const size_t fixed = (size_t)NR * q4_xpitch(p->kr) * 2 + (size_t)2 * Q4_WARPS * NT * 512 +
                         (p->split > 1 ? (size_t)Q4_PART_TILES * NT * 512 : 0);
    if (fixed + (size_t)Q4_WARPS * 2 * slot > Q4_SMEM) continue;
    const int ring = (int)((Q4_SMEM - fixed) / ((size_t)Q4_WARPS * slot));
    // a shallow ring starves the stream: split further while that is possible
    if (ring < 4 && p->split < Q4_MAX_SPLIT && !ln) continue;
    p->ring = ring < Q4_MAX_RING ? ring : Q4_MAX_RING;
    p->smem = fixed + (size_t)Q4_WARPS * p->ring * slot;
    break;
  }
  if (p->split > Q4_MAX_SPLIT) return false;
  const int slots = num_sms() / p->split;
  long best = -1;
  const int st = (p->kr + Q4_STAGE - 1) / Q4_STAGE;
  for (int ks = 1; ks <= Q4_WARPS; ks *= 2) {
    const int gpb = Q4_WARPS / ks;
    const long passes = (ntiles + (long)slots * gpb - 1) / ((long)slots * gpb);
    const long cost = passes * ((st + ks - 1) / ks + 2);
    if (best < 0 || cost < best) {
      best = cost;
      p->ks = ks;
    }
  }
  const int gpb = Q4_WARPS / p->ks;
  int blocks = (ntiles + gpb - 1) / gpb;
  if (blocks > slots) blocks = slots;
  p->grid = blocks * p->split;
  return true;
}

template <int NT, int G>
int q4_launch(Q4Args& a, const Q4Plan& p, cudaStream_t st) {
  CUDA_TRY(once_per_device((const void*)q4_gemv_kernel<NT, G>, [](int) {
    return cudaFuncSetAttribute(q4_gemv_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q4_SMEM);
  }));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(Q4_WARPS * 32);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, q4_gemv_kernel<NT, G>, a));
  LAUNCH_CHECK();
  return GPT2_OK;
}

int q4_run(Q4Args& a, int group, cudaStream_t st) {
  Q4Plan p;
  if (!q4_plan(a.rows, a.N, a.K, group, a.ln != 0, &p)) return GPT2_ERR_UNSUPPORTED_SHAPE;
  a.ks = p.ks; a.split = p.split; a.kr = p.kr; a.ring = p.ring;
  if (a.rows <= 8) {
    if (group == 32) return q4_launch<1, 32>(a, p, st);
    if (group == 64) return q4_launch<1, 64>(a, p, st);
    return q4_launch<1, 128>(a, p, st);
  }
  if (group == 32) return q4_launch<2, 32>(a, p, st);
  if (group == 64) return q4_launch<2, 64>(a, p, st);
  return q4_launch<2, 128>(a, p, st);
}

// (K: at most 65535 k blocks of a grid)
bool q4_shape_ok(int N, int K, int group) {
  return K <= 65535 * QZ_K && (group == 32 || group == 64 || group == 128) && N >= 0 && K >= 1 && K % group == 0;
}

}  // namespace

long q4_pitch(int N) { return ((long)N + 7) & ~7l; }

int q4_quantize(const void* w, int w_f32, long ldw, int N, int K, int group, uint8_t* packed, uint16_t* scales,
                cudaStream_t st) {
  const long pitch = q4_pitch(N);
  bf16* sc = reinterpret_cast<bf16*>(scales);
  const dim3 grid((N + QZ_ROWS - 1) / QZ_ROWS, (K + QZ_K - 1) / QZ_K);
#define QZ(T, G)                                                                                                     \
  CUDA_TRY(launch_k(q4_quantize_kernel<T, G>, grid, 256, 0, st, reinterpret_cast<const T*>(w), ldw, N, K, packed, sc, \
                    pitch))
  if (w_f32) {
    if (group == 32) QZ(float, 32);
    else if (group == 64) QZ(float, 64);
    else QZ(float, 128);
  } else {
    if (group == 32) QZ(bf16, 32);
    else if (group == 64) QZ(bf16, 64);
    else QZ(bf16, 128);
  }
#undef QZ
  LAUNCH_CHECK();
  return GPT2_OK;
}

int decode_gemv_q4(const DecodeGemv& g, const uint8_t* packed, const uint16_t* scales, int group, cudaStream_t st) {
  if (g.rows < 1 || g.rows > 16 || g.K % group) return GPT2_ERR_INVALID_ARG;
  if (g.ln && g.K > 2048) return GPT2_ERR_UNSUPPORTED_SHAPE;
  Q4Args a = {};
  a.in = g.in; a.ldi = g.K; a.in_f32 = !g.in_t; a.ln = g.ln;
  a.ln_g = reinterpret_cast<const bf16*>(g.ln_g); a.ln_b = reinterpret_cast<const bf16*>(g.ln_b);
  a.W = packed; a.sc = reinterpret_cast<const bf16*>(scales); a.pitch = q4_pitch(g.N);
  a.bias = reinterpret_cast<const bf16*>(g.bias);
  a.out = g.out; a.ldo = g.ldo; a.rows = g.rows; a.N = g.N; a.K = g.K; a.w_early = 1;
  a.kc = g.kc; a.vc = g.vc; a.pos = g.pos; a.d = g.d; a.H = g.H; a.hd = g.hd; a.max_len = g.max_len;
  switch (g.epi) {
    case DECODE_QKV: a.epi = Q4_QKV; break;
    case DECODE_RESID: a.epi = Q4_RESID; break;
    case DECODE_GELU: a.epi = Q4_GELU; break;
    case DECODE_LOGITS: a.epi = Q4_F32; a.bias = nullptr; break;
    default: return GPT2_ERR_INVALID_ARG;
  }
  return q4_run(a, group, st);
}

extern "C" {

size_t gpt2_op_q4_packed_bytes(int N, int K) {
  if (N < 1 || K < 1 || K % 32) return 0;
  return (size_t)N * K / 2;
}

size_t gpt2_op_q4_scale_count(int N, int K, int group) {
  if (N < 1 || !q4_shape_ok(N, K, group)) return 0;
  return (size_t)(K / group) * q4_pitch(N);
}

int gpt2_op_q4_quantize(const void* w, int w_fp32, int ldw, int N, int K, int group, uint8_t* packed,
                        uint16_t* scales, void* stream) {
  if (!w || !packed || !scales || N < 0 || K < 0 || ldw < K) return GPT2_ERR_INVALID_ARG;
  if (((uintptr_t)w | (uintptr_t)packed | (uintptr_t)scales) & 15) return GPT2_ERR_INVALID_ARG;
  if (!q4_shape_ok(N, K, group) || ldw % 8) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return GPT2_OK;
  return q4_quantize(w, w_fp32, ldw, N, K, group, packed, scales, reinterpret_cast<cudaStream_t>(stream));
}

int gpt2_op_q4_dequantize(const uint8_t* packed, const uint16_t* scales, int N, int K, int group, void* out,
                          int out_fp32, int ldo, void* stream) {
  if (!packed || !scales || !out || N < 0 || K < 0 || ldo < K) return GPT2_ERR_INVALID_ARG;
  if (((uintptr_t)packed | (uintptr_t)scales | (uintptr_t)out) & 15) return GPT2_ERR_INVALID_ARG;
  if (!q4_shape_ok(N, K, group) || ldo % 8) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return GPT2_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long pitch = q4_pitch(N);
  const int shift = group == 32 ? 5 : (group == 64 ? 6 : 7);
  const bf16* sc = reinterpret_cast<const bf16*>(scales);
  const dim3 grid((N + 15) / 16, (K + 255) / 256);
  if (out_fp32)
    CUDA_TRY(launch_k(q4_dequantize_kernel<float>, grid, 256, 0, st, packed, sc, pitch, shift, N, K,
                      reinterpret_cast<float*>(out), (long)ldo));
  else
    CUDA_TRY(launch_k(q4_dequantize_kernel<bf16>, grid, 256, 0, st, packed, sc, pitch, shift, N, K,
                      reinterpret_cast<bf16*>(out), (long)ldo));
  LAUNCH_CHECK();
  return GPT2_OK;
}

int gpt2_op_gemv_q4(const uint16_t* x, int ldx, const uint8_t* packed, const uint16_t* scales, const uint16_t* bias,
                    void* out, int out_fp32, int ldo, int rows, int N, int K, int group, void* stream) {
  if (!x || !packed || !scales || !out || rows < 0 || rows > 16 || N < 0 || K < 0 || ldx < K || ldo < N)
    return GPT2_ERR_INVALID_ARG;
  if ((((uintptr_t)x | (uintptr_t)packed | (uintptr_t)scales) & 15) || ((uintptr_t)bias & 1) ||
      ((uintptr_t)out & (out_fp32 ? 3 : 1)))
    return GPT2_ERR_INVALID_ARG;
  if (!q4_shape_ok(N, K, group) || K > Q4_MAX_K || ldx % 8) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || N == 0) return GPT2_OK;
  Q4Args a = {};
  a.in = x; a.ldi = ldx;
  a.W = packed; a.sc = reinterpret_cast<const bf16*>(scales); a.pitch = q4_pitch(N);
  a.bias = reinterpret_cast<const bf16*>(bias);
  a.out = out; a.ldo = ldo; a.epi = out_fp32 ? Q4_F32 : Q4_BF16;
  a.rows = rows; a.N = N; a.K = K;
  return q4_run(a, group, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
