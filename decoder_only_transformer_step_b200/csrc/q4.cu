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
// and leave as runs of 32 columns.  HBM asks for 2 or 4 bytes a weight in and
// half a byte out, but the rounding takes longer: bf16, 50304 x 1600, groups of
// 32: 69 us, 46 % of the measured copy rate, issue slots 75 % and ALU pipe 66 % busy.
constexpr int QZ_ROWS = 32, QZ_K = 256;

// q + 8 of eight weights as nibbles, q = clamp(rint(w / s), -7, 7) with the
// division as IEEE rounds it, r an approximate reciprocal of s (2 units in the
// last place).  w r is within 7 * 2^-21 < 1e-5 of the quotient, so its nearest
// integer can be another one only within that of a half: where the distance
// from the integer is above 0.49999 (or a NaN) the division is made.  The
// integers come out of the low bits of w r + 1.5 * 2^23.
DEVI uint32_t q4_word(const float (&w)[8], float s, float r) {
  constexpr float MAGIC = 12582912.f + 8.f;  // bits 0x4b400008
  if (s == 0.f) return 0x88888888u;
  float far = 0.f, d[8];
  uint32_t word = 0;
#pragma unroll
  for (int e = 7; e >= 0; --e) {
    const float t = __fmaf_rn(w[e], r, MAGIC);
    d[e] = fabsf(__fmaf_rn(w[e], r, -__fsub_rn(t, MAGIC)));
    far = d[e] < 0.49999f ? far : 1.f;
    word = word * 16u + __float_as_uint(t);
  }
  word -= 0x4b400000u * 0x11111111u;
  // (a subnormal s can be so coarse that a quotient passes 7: with the others)
  if (far == 0.f && s >= 0x1p-100f) return word;
  const bool all = !(s >= 0x1p-100f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (all || !(d[e] < 0.49999f)) {
      const int q = __float2int_rn(fminf(fmaxf(rintf(w[e] / s), -7.f), 7.f));
      word = (word & ~(15u << (4 * e))) | ((uint32_t)(q + 8) << (4 * e));
    }
  }
  return word;
}

// The same for bf16 weights, whose quotients by a bf16 s are either halves
// exactly or at least 2^-13 from them: the nearest integer of w r is right
// except at exact halves, where the exact remainder w - s q is s / 2 and the
// even neighbour is taken.  (About every second warp meets one: no division.)
DEVI uint32_t q4_word_bf16(const float (&w)[8], float s, float r) {
  constexpr float MAGIC = 12582912.f + 8.f;
  const float hs = 0.5f * s;
  float rem[8];
  uint32_t word = 0;
#pragma unroll
  for (int e = 7; e >= 0; --e) {
    const float t = __fmaf_rn(w[e], r, MAGIC);
    rem[e] = __fmaf_rn(-s, __fsub_rn(t, MAGIC), w[e]);
    word = word * 16u + __float_as_uint(t);
  }
  word -= 0x4b400000u * 0x11111111u;
  float far = fmaxf(fabsf(rem[0]), fabsf(rem[1]));
#pragma unroll
  for (int e = 2; e < 8; e += 2)
    asm("max.f32 %0, %0, %1, %2;" : "+f"(far) : "f"(fabsf(rem[e])), "f"(fabsf(rem[e + 1])));
  if (far == hs) {
    const uint32_t odd = word;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(rem[e]) == hs && (odd & (1u << (4 * e)))) word += rem[e] > 0.f ? 1u << (4 * e) : 0u - (1u << (4 * e));
  }
  return word;
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
  constexpr int W4 = sizeof(T) / 2;  // 16-byte words of eight weights
  uint4 raw[4][W4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + warp * 4 + i;
#pragma unroll
    for (int h = 0; h < W4; ++h)
      raw[i][h] = n < N && k < K ? reinterpret_cast<const uint4*>(w + (size_t)n * ldw + k)[h] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the largest magnitude as an unsigned integer: NaN above infinity above
    // every finite value, so that a group holding either gets such a scale
    uint32_t top;
    float v[8];
    if constexpr (sizeof(T) == 2) {
      const uint4 u = raw[i][0];
      top = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
      top = max(top & 0xffff0000u, top << 16);
      v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
      v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
    } else {
      const uint32_t x[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                             raw[i][W4 - 1].x, raw[i][W4 - 1].y, raw[i][W4 - 1].z, raw[i][W4 - 1].w};
      top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        top = max(top, x[e] & 0x7fffffffu);
        v[e] = __uint_as_float(x[e]);
      }
    }
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // (a bf16 over 7 is never within 2^-12 of a bf16 rounding border: the product with 1/7 rounds alike)
    const bf16 sb = __float2bfloat16_rn(sizeof(T) == 2 ? __uint_as_float(top) * (1.f / 7.f) : __uint_as_float(top) / 7.f);
    const float s = __bfloat162float(sb);
    const int n = n0 + warp * 4 + i;
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    // (a tiny, NaN or infinite s goes the careful way)
    const uint32_t word = sizeof(T) == 2 && s >= 0x1p-100f && s < 0x1p100f ? q4_word_bf16(v, s, r) : q4_word(v, s, r);
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

DEVI uint32_t q4_mul2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
DEVI uint32_t q4_sub136(uint32_t a) {
  const uint32_t c = 0x43084308u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The values the nibbles stand for, s q (exact in fp32, rounded once to bf16
// where T is bf16).  A warp takes 256 inputs of 8 rows, a lane 8 inputs of
// each with all loads in flight together; the 64 rows of a block share the
// sectors of the scales.  Bound by HBM, mostly its writes: bf16, 50304 x 1600:
// 206 MB in 37 us, 86 % of the measured copy rate.
constexpr int DQ_ROWS = 8;
template <typename T>
__global__ void __launch_bounds__(256)
    q4_dequantize_kernel(const uint8_t* packed, const bf16* scales, long pitch, int group_shift, int N, int K,
                         T* __restrict__ out, long ldo) {
  pdl_start();
  const int k = (blockIdx.y * 32 + (threadIdx.x & 31)) * 8;
  if (k >= K) return;
  const int n0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * DQ_ROWS;
  if (n0 >= N) return;
  uint32_t w[DQ_ROWS];
  // the eight rows' scales lie side by side (n0 and the pitch are multiples of 8)
  const uint4 s8 = *reinterpret_cast<const uint4*>(scales + (size_t)(k >> group_shift) * pitch + n0);
#pragma unroll
  for (int i = 0; i < DQ_ROWS; ++i)
    w[i] = *reinterpret_cast<const uint32_t*>(packed + ((size_t)min(n0 + i, N - 1) * K + k) / 2);
  const float s[DQ_ROWS] = {bf16lo(s8.x), bf16hi(s8.x), bf16lo(s8.y), bf16hi(s8.y),
                            bf16lo(s8.z), bf16hi(s8.z), bf16lo(s8.w), bf16hi(s8.w)};
#pragma unroll
  for (int i = 0; i < DQ_ROWS; ++i) {
    if (n0 + i >= N) break;
    T* p = out + (size_t)(n0 + i) * ldo + k;
    // nibbles e and e + 4 as bf16: bits 0x4300 | nibble are 128 + nibble
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = q4_sub136((w[i] >> (4 * e)) & 0x000f000fu | 0x43004300u);
    if constexpr (sizeof(T) == 2) {
      const uint32_t s2 = __float_as_uint(s[i]) >> 16 | __float_as_uint(s[i]);
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = q4_mul2(q[e], s2);
      *reinterpret_cast<uint4*>(p) = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                                __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(s[i] * bf16lo(q[0]), s[i] * bf16lo(q[1]), s[i] * bf16lo(q[2]), s[i] * bf16lo(q[3]));
      *reinterpret_cast<float4*>(p + 4) =
          make_float4(s[i] * bf16hi(q[0]), s[i] * bf16hi(q[1]), s[i] * bf16hi(q[2]), s[i] * bf16hi(q[3]));
    }
  }
}

// ------------------------------------------------- matrix-vector products --
// Bound by HBM reads of the nibbles, and next to that by the instructions that
// bring them to the products: at the copy bandwidth 13e12 weights/s leave an
// SM's four schedulers about three instructions for 32 weights.  So the
// products run on mma.sync m16n8k16 with the weights as A (16 output columns
// a warp tile) and the rows of x as B, and a nibble is not converted at all: a
// bf16 whose upper byte is zero is its lower byte times 2^-133 (subnormal
// numbers and the lowest normal ones lie on one line), which mma takes
// exactly, so that one AND leaves two operands (a nibble in the upper half of
// a byte counts 16-fold).  To match, each row of x is staged times the power
// of two that brings its largest magnitude to 2^114, a sixteenth of that at
// odd k: exact in bf16, but for numbers below 2^-234 of the row's largest.
// So a row's sum is formed in a unit of at most 2^19 of its largest magnitude:
// with |q| <= 8 and 2^15 inputs it stays below any scale's own bound (no sum
// overflows that the result does not), and it is subnormal, off by up to
// 2^-131 of that magnitude an addition, only where scales are below 2^-100.
// The nibbles are q + 8, so a group's sum starts at -8 sum x instead of 0 (the
// group sums of x are formed once, when x is staged).  A group's products are
// summed in fp32 by the tensor core and multiplied by the group's scale in
// fp32: no weight is rounded again.
//
// A lane's share of a stage's row is what its quad's mma need of one group at a
// time: 16, 8 or 4 bytes for groups of 128, 64 or 32, so that a product never
// crosses a group; the order of the inputs inside a group is the lanes' own,
// and x is staged in it.
//
// A block is 16 warps.  KS of them share a tile of 16 columns, each taking
// every KS-th stage of 256 inputs; their sums meet in shared memory in a fixed
// order.  Each warp copies its own stages (16 rows x 128 bytes and their
// scales) into a ring of its own with cp.async, several ahead, across tile
// borders: no block-wide wait stands in the stream.  Inputs too long for
// shared memory are split over the blocks of a cluster (up to 8), whose sums
// meet through distributed shared memory, again in a fixed order (the rows in
// two or three groups, each a pass over the weights, instead: groups of 128, 16
// x 50304 x 6400 75 us, split 71; 5 x 28673 x 16384 110, 60).
//
// 8 x 50304 x 1600, groups of 32: 18 us (2.6 TB/s); 5 x 28673 x 8192, groups of
// 128: 33 us (3.6 TB/s, 27.6 without the products): half the issue slots and
// ALU cycles taken (48 and 51 %, 36 and 45 %), the rest waits of 16 warps.
constexpr int Q4_WARPS = 16;
constexpr int Q4_COLS = 16;                    // output columns of a tile (the mma M)
constexpr int Q4_STAGE = 256;                  // inputs of a stage
constexpr int Q4_RP = Q4_STAGE / 2;            // bytes of a staged row
constexpr int Q4_MAX_SPLIT = 8;
constexpr int Q4_PART_TILES = 8;               // tiles whose sums a cluster exchanges at once (1 where that does not fit)
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
  int ks, split, kr, ring, part, w_early, wpr;  // wpr: warps of a row of x while it is staged
  void* kc;
  void* vc;
  const int32_t* pos;
  int d, H, hd, max_len;
};
enum Q4Epi : int { Q4_BF16 = 0, Q4_F32, Q4_QKV, Q4_RESID, Q4_GELU };

// Shared memory of a block, in bytes: the rows of x, the group sums, the row
// factors, the warps' sums, the cluster's, the rings.
__host__ __device__ inline int q4_xpitch(int kr) { return kr % 64 ? kr : kr + 32; }  // an odd multiple of 64 bytes
__host__ __device__ constexpr int q4_slot(int group) { return Q4_COLS * Q4_RP + Q4_STAGE / group * Q4_COLS * 2; }
// Where 16-byte piece c of staged row r lies: the pieces are exchanged so that
// the lanes' 16-, 8- or 4-byte reads of 2, 4 or 8 rows fall into different banks.
template <int G> DEVI int q4_piece(int r, int c) {
  constexpr int W = G / 32;
  return c ^ ((r & (8 / W - 1)) * W);
}
struct Q4Smem {
  int xg, fac, red, part, ring;
};
__host__ __device__ inline Q4Smem q4_smem(int nr, int rows, int kr, int group, int part_tiles) {
  Q4Smem m;
  m.xg = rows * q4_xpitch(kr) * 2;
  m.fac = m.xg + ((kr / group * nr * 4 + 15) & ~15);
  m.red = m.fac + 16 * 8;
  m.part = m.red + Q4_WARPS * (nr / 8) * 512;
  m.ring = m.part + part_tiles * (nr / 8) * 512;
  return m;
}

DEVI void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
DEVI void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest ring - 2 groups have landed (rings of 2, 3 and 4 slots).
DEVI void cp_wait_ring(int ring) {
  if (ring == 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (ring == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// a lane's W words of a group (W 4, 2 or 1)
template <int W> DEVI void lds_words(uint32_t a, uint32_t (&v)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a) : "memory");
}
DEVI float2 lds64f(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
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
DEVI void q4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
DEVI float4 q4_ld4(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}
DEVI uint4 q4_pack8(const float4& a, const float4& b) {
  return make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
}

DEVI uint32_t q4_max2(uint32_t m, const uint4& v) {
  return __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
}

// Inputs [k0, k0 + kn) of the rows -> xs [rows][xp] and the rows' factors
// (the power of two that undoes the scaling and the 2^-133, as two floats).
// wpr warps share a row (their number a power of two, the rows' times it at
// most 16); a lane holds its units of 8 inputs in registers from the load to
// the scaled store.  Rows past a.rows are not written: what the mma make of
// them stays in columns that are dropped.  All threads call it.
template <int G>
DEVI void q4_stage_x(const Q4Args& a, bf16* xs, int xp, float2* fac, uint32_t* wmax, int k0, int kn, int warp, int lane) {
  constexpr int U = 8;  // units a lane holds at once
  constexpr int W = G / 32;
  const int wpr = a.wpr, r = warp / wpr, part = warp % wpr, n8 = kn / 8, mine = (n8 + wpr - 1 - part) / wpr;
  // (unit j of this warp's lane: part + wpr * (lane + 32 u))
  const bool live = r < a.rows;
  uint4 v[U];
  float mu = 0.f, rs = 0.f;
  if (a.ln && live) {
    // (K <= 2048, one chunk.)  Every warp of the row forms its two statistics.
    const float* src = reinterpret_cast<const float*>(a.in) + (size_t)r * a.ldi;
    float s = 0.f, q = 0.f;
#pragma unroll 8
    for (int i = lane; i < 2 * n8; i += 32) {
      const float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
      s += (f.x + f.y) + (f.z + f.w);
    }
    mu = warp_sum(s) / a.K;
#pragma unroll 8
    for (int i = lane; i < 2 * n8; i += 32) {
      const float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
      const float t0 = f.x - mu, t1 = f.y - mu, t2 = f.z - mu, t3 = f.w - mu;
      q += (t0 * t0 + t1 * t1) + (t2 * t2 + t3 * t3);
    }
    rs = rsqrtf(warp_sum(q) / a.K + 1e-5f);
  }
  auto load = [&](int j) -> uint4 {
    const int k = k0 + 8 * (part + wpr * j);
    if (a.ln) {
      const float* p = reinterpret_cast<const float*>(a.in) + (size_t)r * a.ldi + k;
      float4 o[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = *reinterpret_cast<const float4*>(p + 4 * h);
        const float4 gg = q4_ld4(a.ln_g + k + 4 * h), bb = q4_ld4(a.ln_b + k + 4 * h);
        o[h] = make_float4((x.x - mu) * rs * gg.x + bb.x, (x.y - mu) * rs * gg.y + bb.y, (x.z - mu) * rs * gg.z + bb.z,
                           (x.w - mu) * rs * gg.w + bb.w);
      }
      return q4_pack8(o[0], o[1]);
    }
    if (a.in_f32) {
      const float* p = reinterpret_cast<const float*>(a.in) + (size_t)r * a.ldi + k;
      return q4_pack8(*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4));
    }
    return *reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.in) + (size_t)r * a.ldi + k);
  };
  // the row's largest magnitude, as the bits of a bf16
  uint32_t m2 = 0;
  if (live) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (lane + 32 * u < mine) v[u] = load(lane + 32 * u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m2 = q4_max2(m2, v[u]);
    for (int j = lane + 32 * U; j < mine; j += 32) m2 = q4_max2(m2, load(j));  // (very long rows: loaded again below)
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
  if (wpr > 1) {
    if (lane == 0) wmax[warp] = m;
    __syncthreads();
    m = wmax[lane < wpr ? r * wpr + lane : r * wpr];
    m = __reduce_max_sync(0xffffffffu, m);
  }
  if (!live) return;
  // 2^114 over the power of two at or below it (1 for a row of zeros, and for
  // one that holds an infinity or NaN: its sums are not finite anyway), a
  // sixteenth of it in the upper halves, the odd inputs; in two steps where
  // that is above 2^127
  const int ex = (int)(m >> 7), sh = m == 0 || ex == 255 ? 0 : 241 - ex, s1 = sh > 127 ? sh - 127 : 0, s2 = sh - s1;
  const uint32_t f1 = (uint32_t)(127 + s1) * 0x00800080u, f2 = (uint32_t)(127 + s2) << 7 | (uint32_t)(123 + s2) << 23;
  if (lane == 0 && part == 0) {
    const int un = 133 - sh;
    fac[r] = make_float2(__int_as_float((127 + un / 2) << 23), __int_as_float((127 + (un - un / 2)) << 23));
  }
  auto store = [&](int j, uint4 x) {
    const int i = part + wpr * j;
    if (s1) x = make_uint4(q4_mul2(x.x, f1), q4_mul2(x.y, f1), q4_mul2(x.z, f1), q4_mul2(x.w, f1));
    x = make_uint4(q4_mul2(x.x, f2), q4_mul2(x.y, f2), q4_mul2(x.z, f2), q4_mul2(x.w, f2));
    // in the order in which the nibbles of a word unpack (0 4 1 5 2 6 3 7);
    // unit c of lane t in its group goes to place 4 c + t: a quad's reads are consecutive
    const int in_g = i % (4 * W), at = i - in_g + 4 * (in_g % W) + in_g / W;
    *reinterpret_cast<uint4*>(xs + (size_t)r * xp + 8 * at) =
        make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                   __byte_perm(x.y, x.w, 0x7632));
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (lane + 32 * u < mine) store(lane + 32 * u, v[u]);
  for (int j = lane + 32 * U; j < mine; j += 32) store(j, load(j));
}

// The epilogue's operands of one lane, loaded ahead of the products: the
// biases of columns n0 + g and n0 + g + 8, the old residuals.
template <int NT> struct Q4Pre {
  float b[2], x[NT][4];
};
template <int NT> DEVI void q4_preload(const Q4Args& a, Q4Pre<NT>& p, int n0, int g, int t) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + g + 8 * h;
    p.b[h] = a.bias && n < a.N ? to_f(a.bias[n]) : 0.f;
  }
  if (a.epi == Q4_RESID) {
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + g + 8 * (i >> 1), r = 8 * m + 2 * t + (i & 1);
        p.x[m][i] = n < a.N && r < a.rows ? reinterpret_cast<const float*>(a.out)[(size_t)r * a.ldo + n] : 0.f;
      }
  }
}
// One lane's four sums of n-tile m: columns n0 + g, n0 + g + 8 (values 0 1,
// 2 3), rows 8 m + 2 t and the next (values 0 2, 1 3).
template <int NT> DEVI void q4_epilogue(const Q4Args& a, const float4& s, const Q4Pre<NT>& p, int m, int n0, int g, int t) {
  const float v4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + g + 8 * (i >> 1), r = 8 * m + 2 * t + (i & 1);
    if (n >= a.N || r >= a.rows) continue;
    const float v = v4[i] + p.b[i >> 1];
    const size_t at = (size_t)r * a.ldo + n;
    float* of = reinterpret_cast<float*>(a.out);
    bf16* ob = reinterpret_cast<bf16*>(a.out);
    switch (a.epi) {
      case Q4_BF16: ob[at] = from_f<bf16>(v); break;
      case Q4_F32: of[at] = v; break;
      case Q4_RESID: of[at] = p.x[m][i] + v; break;
      case Q4_GELU: ob[at] = from_f<bf16>(gelu_f<false>(v)); break;
      default: {  // Q4_QKV: q to out, k and v into the cache at pos[r]
        if (n < a.d) {
          of[at] = v;
        } else {
          const int kind = n >= 2 * a.d, nn = n - a.d - kind * a.d, ps = a.pos[r];
          if (ps >= 0 && ps < a.max_len) {
            bf16* plane = reinterpret_cast<bf16*>(kind ? a.vc : a.kc);
            plane[(((size_t)r * a.H + nn / a.hd) * a.max_len + ps) * a.hd + nn % a.hd] = from_f<bf16>(v);
          }
        }
      }
    }
  }
}

template <int NT, int G>
__global__ void __launch_bounds__(Q4_WARPS * 32, 1) q4_gemv_kernel(const __grid_constant__ Q4Args a) {
  extern __shared__ __align__(128) uint8_t q4_smem_buf[];
  __shared__ uint32_t wmax[Q4_WARPS];
  constexpr int NR = 8 * NT;            // rows of x held
  constexpr int SLOT = q4_slot(G), RP = Q4_RP;
  constexpr int GS = Q4_STAGE / G;      // groups of a stage
  constexpr int W = G / 32;             // words a lane has of a group
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = a.split > 1 ? (int)cluster_ctarank() : 0;
  const int bx = blockIdx.x / a.split, gx = gridDim.x / a.split;
  const int k0 = rank * a.kr, kn = max(0, min(a.kr, a.K - k0));
  const int xp = q4_xpitch(a.kr);
  const Q4Smem sm = q4_smem(NR, a.rows, a.kr, G, a.part);
  bf16* xs = reinterpret_cast<bf16*>(q4_smem_buf);
  float* xg = reinterpret_cast<float*>(q4_smem_buf + sm.xg);
  float2* fac = reinterpret_cast<float2*>(q4_smem_buf + sm.fac);
  float4* red = reinterpret_cast<float4*>(q4_smem_buf + sm.red);    // [warps][NT][32]
  float4* part = reinterpret_cast<float4*>(q4_smem_buf + sm.part);  // (split) [tiles][NT][32]
  const uint32_t ring = smem_u32(q4_smem_buf) + sm.ring + warp * a.ring * SLOT;
  const uint32_t ring_end = ring + a.ring * SLOT;
  const int ks = a.ks, grp = warp / ks, si = warp % ks, gpb = Q4_WARPS / ks;
  const int ntiles = (a.N + Q4_COLS - 1) / Q4_COLS, nst = (kn + Q4_STAGE - 1) / Q4_STAGE;
  // pass p of this block: its group's tile is (p gpb + grp) gx + bx, so that
  // every block has the same number of tiles, give or take one
  const int tstep = gx * gpb;

  // the producer side of this warp's ring: the next stage's sources (16 bytes
  // of four rows of nibbles a lane, 16 bytes of scales), its tile and place
  const int nfull = kn / Q4_STAGE;
  int pt = si < nst ? grp * gx + bx : ntiles, ps = si;
  uint32_t pslot = ring;
  const int prow = lane >> 3, pc = lane & 7;
  uint32_t dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = (prow + 4 * i) * RP + 16 * q4_piece<G>(prow + 4 * i, pc);
  const uint32_t dsc = Q4_COLS * RP + lane * 16;
  const uint8_t* w[4] = {nullptr, nullptr, nullptr, nullptr};
  const bf16* scp = nullptr;
  bool sc_live = false;
  auto tile_sources = [&]() {
    const int n0 = pt * Q4_COLS, kk = k0 + ps * Q4_STAGE;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // columns past N read the last one and are dropped
      w[i] = a.W + ((size_t)min(n0 + prow + 4 * i, a.N - 1) * a.K + kk) / 2 + 16 * pc;
    // 16 columns of scales a group, 8 a copy (the pitch is a multiple of 8)
    const int c = n0 + 8 * (lane & 1);
    sc_live = lane < 2 * GS && c < a.pitch;
    scp = a.sc + (size_t)(kk / G + (lane >> 1)) * a.pitch + c;
  };
  if (pt < ntiles) tile_sources();
  const size_t sc_step = (size_t)ks * GS * a.pitch;
  const int w_step = ks * Q4_RP;
  auto issue = [&]() {
    if (pt < ntiles) {
      if (ps < nfull) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(pslot + dw[i], w[i]);
        if (sc_live) cp_async16(pslot + dsc, scp);
      } else {
        const int left = kn - nfull * Q4_STAGE;  // (a multiple of 32 and of G)
        if (pc < left / 32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async16(pslot + dw[i], w[i]);
        }
        if (sc_live && (lane >> 1) * G < left) cp_async16(pslot + dsc, scp);
      }
      ps += ks;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] += w_step;
      scp += sc_step;
      if (ps >= nst) {
        ps = si;
        pt += tstep;
        if (pt < ntiles) tile_sources();
      }
    }
    cp_commit();
    pslot = pslot + SLOT == ring_end ? ring : pslot + SLOT;
  };

  pdl_trigger();
  // In the decode step no kernel writes weights and its first kernel lets its
  // successors start only after every kernel before the step has finished:
  // there (w_early) the first stages are requested before the wait.
  if (!a.w_early) pdl_wait();
  for (int i = 0; i < a.ring - 1; ++i) issue();
  if (a.w_early) pdl_wait();
  q4_stage_x<G>(a, xs, xp, fac, wmax, k0, kn, warp, lane);
  __syncthreads();
  // this lane's rows of x (those past the last are not staged: the last one again, dropped)
  uint32_t xrow[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) xrow[m] = smem_u32(xs) + (uint32_t)(min(g + 8 * m, a.rows - 1) * xp * 2 + 16 * t);
  // -8 times the group sums: mma with every weight -8 (bits 0x8008, in the
  // upper halves of bytes 0x8080)
  for (int j = warp; j < kn / G; j += Q4_WARPS) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const uint4 xv = lds128(xrow[m] + 64 * (W * j + c));
        q4_mma(d, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, xv.x, xv.y);
        q4_mma(d, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, xv.z, xv.w);
      }
      if (g == 0) *reinterpret_cast<float2*>(xg + j * NR + 8 * m + 2 * t) = make_float2(d[0], d[1]);
    }
  }
  __syncthreads();

  const uint32_t xgb = smem_u32(xg) + (uint32_t)(2 * t * 4);
  const uint32_t sw = 16 * q4_piece<G>(g, 0);
  uint32_t cslot = ring;
  float acc[NT][4];
  // the products of groups [0, ng) of the stage in cslot, stage s of the k range
  auto stage = [&](int s, int ng) {
    const uint32_t w = cslot + g * RP;
    const uint32_t sc = cslot + Q4_COLS * RP + 2 * g;
    const uint32_t xgk = xgb + s * GS * NR * 4;
    uint32_t xk[NT];
#pragma unroll
    for (int m = 0; m < NT; ++m) xk[m] = xrow[m] + s * Q4_STAGE * 2;
#pragma unroll
    for (int j = 0; j < GS; ++j) {
      if (j < ng) {
        // a second chain of sums where a lane has several words of a group
        float c0[NT][4], c1[NT][4];
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const float2 x8 = lds64f(xgk + (j * NR + 8 * m) * 4);
          c0[m][0] = c0[m][2] = x8.x;
          c0[m][1] = c0[m][3] = x8.y;
          c1[m][0] = c1[m][1] = c1[m][2] = c1[m][3] = 0.f;
        }
        uint32_t wa[W], wb[W];
        // (the pieces of rows g and g + 8 are exchanged alike)
        const uint32_t at = ((16 * W * j) ^ sw) + 4 * W * t;
        lds_words<W>(w + at, wa);
        lds_words<W>(w + 8 * RP + at, wb);
#pragma unroll
        for (int c = 0; c < W; ++c) {
          constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;
          const uint32_t va = wa[c] >> 8, vb = wb[c] >> 8;
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            const uint4 xv = lds128(xk[m] + 64 * (W * j + c));
            q4_mma(c0[m], wa[c] & LO, wb[c] & LO, wa[c] & HI, wb[c] & HI, xv.x, xv.y);
            q4_mma(W > 1 ? c1[m] : c0[m], va & LO, vb & LO, va & HI, vb & HI, xv.z, xv.w);
          }
        }
        const float s0 = lds_bf16(sc + 32 * j), s1 = lds_bf16(sc + 32 * j + 16);
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[m][i] = fmaf(i < 2 ? s0 : s1, W > 1 ? c0[m][i] + c1[m][i] : c0[m][i], acc[m][i]);
      }
    }
  };
  int it = 0;
  const int ptg = max(1, a.part / gpb);  // (split) tile passes between exchanges
  for (int base = bx; base < ntiles; base += tstep) {
    const int tile = base + grp * gx;
    const bool joins = si == it % ks;  // the warps of a tile take turns at its epilogue
    Q4Pre<NT> pre;
    if (joins && a.split == 1) q4_preload<NT>(a, pre, tile * Q4_COLS, g, t);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    if (tile < ntiles) {
      for (int s = si; s < nst; s += ks) {
        cp_wait_ring(a.ring);
        __syncwarp();  // every lane's copies of this stage have landed; the slot before it is free
        issue();
        if (s < nfull) stage(s, GS);
        else stage(s, (kn - nfull * Q4_STAGE) / G);
        cslot = cslot + SLOT == ring_end ? ring : cslot + SLOT;
      }
    }
    // the tile's warps meet: once all are here the sums of the last tile have been read
    float4 tot[NT];
    if (ks > 1) {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(ks * 32) : "memory");
#pragma unroll
      for (int m = 0; m < NT; ++m)
        red[(warp * NT + m) * 32 + lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(ks * 32) : "memory");
    }
    if (joins) {
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        if (ks > 1) {
          tot[m] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int x = 0; x < ks; ++x) {
            const float4 q = red[((grp * ks + x) * NT + m) * 32 + lane];
            tot[m].x += q.x;
            tot[m].y += q.y;
            tot[m].z += q.z;
            tot[m].w += q.w;
          }
        } else {
          tot[m] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        }
        // out of the row's scaling and the nibbles' 2^-133
        const float2 fa = fac[8 * m + 2 * t], fb = fac[8 * m + 2 * t + 1];
        tot[m].x = tot[m].x * fa.x * fa.y;
        tot[m].y = tot[m].y * fb.x * fb.y;
        tot[m].z = tot[m].z * fa.x * fa.y;
        tot[m].w = tot[m].w * fb.x * fb.y;
        if (a.split == 1 && tile < ntiles) q4_epilogue<NT>(a, tot[m], pre, m, tile * Q4_COLS, g, t);
      }
    }
    if (a.split > 1) {
      // tiles of this block since the last exchange: slot (pass, group)
      const int pass = it % ptg;
      if (joins)
#pragma unroll
        for (int m = 0; m < NT; ++m) part[((pass * gpb + grp) * NT + m) * 32 + lane] = tot[m];
      const bool last = base + tstep >= ntiles;
      if (pass == ptg - 1 || last) {
        cluster_sync_all();
        // slot x is finished by rank x % split, one warp a slot
        const int pbase = base - pass * tstep, nslots = (pass + 1) * gpb;
        for (int x = rank + warp * a.split; x < nslots; x += Q4_WARPS * a.split) {
          const int tl = pbase + x * gx;
          if (tl < ntiles) {
            q4_preload<NT>(a, pre, tl * Q4_COLS, g, t);
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
              q4_epilogue<NT>(a, sum, pre, m, tl * Q4_COLS, g, t);
            }
          }
        }
        cluster_sync_all();  // the slots are free again, and no block leaves while another reads it
      }
    }
    ++it;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The same products for few tiles, where the time is that of one round trip to
// memory and not of the stream: staging x, which pays off over many tiles of
// a block, would cost more than it saves.  A block of 16 warps takes one
// tile of 16 columns, its warps every 16th unit of max(G, 64) inputs; nibbles
// and x come straight from memory as fragments, a unit ahead.  Here a nibble
// is converted: bf16 bits 0x3e00 | nibble are (128 + nibble) / 1024, and one
// packed subtraction of 136 / 1024 leaves two q / 1024 exactly (a group's sum
// of up to 128 products |q| <= 8 then stays in range whatever x is; the scale
// takes the 1024 back, or the sum where the scale would be infinite: looking
// at the scales costs a decode step of the 124M model 1 to 2 %).  fp32 or LayerNorm'd rows are first
// brought into shared memory as bf16 (STAGED; one warp a row).  1 x 4800 x 1600
// takes 4.9 us, 16 x 1600 x 6400 8.0: bound by waits for memory, at 16 rows by
// every block's own reading of all of x.
constexpr int QD_WARPS = 16;
constexpr int QD_STAGED_K = 2048;  // widest staged row
constexpr int QD_PAD = 32;         // elements behind a staged row: an odd multiple of 64 bytes in all
DEVI uint32_t q4_pair(uint32_t w, int i) {
  const uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x3e003e00u, c = 0x3e083e08u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Row r of the fp32 input, LayerNorm'd if a.ln, as bf16; a whole warp.
DEVI void q4_stage_row(const Q4Args& a, bf16* dst, int r, int lane) {
  const float* src = reinterpret_cast<const float*>(a.in) + (size_t)r * a.ldi;
  const int n4 = a.K / 4;
  float mu = 0.f, rs = 1.f;
  if (a.ln) {
    float s = 0.f, q = 0.f;
#pragma unroll 8
    for (int i = lane; i < n4; i += 32) {
      const float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
      s += (f.x + f.y) + (f.z + f.w);
    }
    mu = warp_sum(s) / a.K;
#pragma unroll 8
    for (int i = lane; i < n4; i += 32) {
      const float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
      const float t0 = f.x - mu, t1 = f.y - mu, t2 = f.z - mu, t3 = f.w - mu;
      q += (t0 * t0 + t1 * t1) + (t2 * t2 + t3 * t3);
    }
    rs = rsqrtf(warp_sum(q) / a.K + 1e-5f);
  }
#pragma unroll 4
  for (int i = lane; i < n4; i += 32) {
    float4 f = *reinterpret_cast<const float4*>(src + 4 * i);
    if (a.ln) {
      const float4 gg = q4_ld4(a.ln_g + 4 * i), bb = q4_ld4(a.ln_b + 4 * i);
      f = make_float4((f.x - mu) * rs * gg.x + bb.x, (f.y - mu) * rs * gg.y + bb.y, (f.z - mu) * rs * gg.z + bb.z,
                      (f.w - mu) * rs * gg.w + bb.w);
    }
    *reinterpret_cast<uint2*>(dst + 4 * i) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
  }
}

template <int NT, int G, bool STAGED>
__global__ void __launch_bounds__(QD_WARPS * 32) q4_direct_kernel(const __grid_constant__ Q4Args a) {
  extern __shared__ __align__(16) uint8_t qd_smem[];  // (STAGED) the rows
  constexpr int W = G / 32;                     // words a lane has of a group
  constexpr int UG = G < 64 ? 2 : 1;            // groups of a unit
  constexpr int UK = UG * G;                    // inputs of a unit
  __shared__ float4 red[QD_WARPS][NT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * Q4_COLS, nun = (a.K + UK - 1) / UK;
  // columns and rows past the last read the last one and are dropped
  const uint8_t* wa = a.W + (size_t)min(n0 + g, a.N - 1) * a.K / 2 + 4 * W * t;
  const uint8_t* wb = a.W + (size_t)min(n0 + g + 8, a.N - 1) * a.K / 2 + 4 * W * t;
  bf16* const xs = reinterpret_cast<bf16*>(qd_smem);
  const bf16* x[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    const size_t r = min(g + 8 * m, a.rows - 1);
    x[m] = (STAGED ? xs + r * (a.K + QD_PAD) : reinterpret_cast<const bf16*>(a.in) + r * a.ldi) + 8 * W * t;
  }
  const bf16* sa = a.sc + min(n0 + g, a.N - 1);
  const bf16* sb = a.sc + min(n0 + g + 8, a.N - 1);
  struct Unit {
    uint32_t wa[UG][W], wb[UG][W];
    uint4 x[NT][UG][W];
    float s0[UG], s1[UG];
  };
  pdl_trigger();
  if (!a.w_early) pdl_wait();
  auto load_w = [&](Unit& u, int i) {
#pragma unroll
    for (int j = 0; j < UG; ++j) {
      const int k = i * UK + j * G;
      const bool in = i < nun && k < a.K;
#pragma unroll
      for (int c = 0; c < W; ++c) u.wa[j][c] = u.wb[j][c] = 0x88888888u;
      u.s0[j] = u.s1[j] = 0.f;
      if (in) {
        if constexpr (W == 4) {
          const uint4 p = *reinterpret_cast<const uint4*>(wa + k / 2), q = *reinterpret_cast<const uint4*>(wb + k / 2);
          u.wa[j][0] = p.x; u.wa[j][1] = p.y; u.wa[j][2] = p.z; u.wa[j][3] = p.w;
          u.wb[j][0] = q.x; u.wb[j][1] = q.y; u.wb[j][2] = q.z; u.wb[j][3] = q.w;
        } else if constexpr (W == 2) {
          const uint2 p = *reinterpret_cast<const uint2*>(wa + k / 2), q = *reinterpret_cast<const uint2*>(wb + k / 2);
          u.wa[j][0] = p.x; u.wa[j][1] = p.y;
          u.wb[j][0] = q.x; u.wb[j][1] = q.y;
        } else {
          u.wa[j][0] = *reinterpret_cast<const uint32_t*>(wa + k / 2);
          u.wb[j][0] = *reinterpret_cast<const uint32_t*>(wb + k / 2);
        }
        u.s0[j] = to_f(sa[(size_t)(k / G) * a.pitch]);
        u.s1[j] = to_f(sb[(size_t)(k / G) * a.pitch]);
      }
    }
  };
  auto load_x = [&](Unit& u, int i) {
#pragma unroll
    for (int j = 0; j < UG; ++j) {
      const int k = i * UK + j * G;
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int c = 0; c < W; ++c)
          u.x[m][j][c] = i < nun && k < a.K ? *reinterpret_cast<const uint4*>(x[m] + k + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  Unit cur, next;
  load_w(cur, warp);
  if (a.w_early) pdl_wait();
  if constexpr (STAGED) {
    for (int r = warp; r < a.rows; r += QD_WARPS) q4_stage_row(a, xs + (size_t)r * (a.K + QD_PAD), r, lane);
    __syncthreads();
  }
  load_x(cur, warp);
  Q4Pre<NT> pre;
  if (warp == 0) q4_preload<NT>(a, pre, n0, g, t);
  float acc[NT][4];
#pragma unroll
  for (int m = 0; m < NT; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
  for (int i = warp; i < nun; i += QD_WARPS) {
    load_w(next, i + QD_WARPS);
    load_x(next, i + QD_WARPS);
#pragma unroll
    for (int j = 0; j < UG; ++j) {
      float c0[NT][4];
#pragma unroll
      for (int m = 0; m < NT; ++m) c0[m][0] = c0[m][1] = c0[m][2] = c0[m][3] = 0.f;
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const uint32_t p = cur.wa[j][c], q = cur.wb[j][c];
        const uint32_t p0 = q4_pair(p, 0), q0 = q4_pair(q, 0), p1 = q4_pair(p, 1), q1 = q4_pair(q, 1);
        const uint32_t p2 = q4_pair(p, 2), q2 = q4_pair(q, 2), p3 = q4_pair(p, 3), q3 = q4_pair(q, 3);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const uint4 v = cur.x[m][j][c];  // into the nibbles' order: 0 4, 1 5, 2 6, 3 7
          q4_mma(c0[m], p0, q0, p1, q1, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
          q4_mma(c0[m], p2, q2, p3, q3, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
      }
      // (a sum that the 1024 makes infinite would be so times a scale above 2^118 too)
      const bool b0 = cur.s0[j] < 0x1p118f, b1 = cur.s1[j] < 0x1p118f;
      const float s0 = b0 ? 1024.f * cur.s0[j] : cur.s0[j], s1 = b1 ? 1024.f * cur.s1[j] : cur.s1[j];
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[m][e] = fmaf(e < 2 ? s0 : s1, (e < 2 ? b0 : b1) ? c0[m][e] : 1024.f * c0[m][e], acc[m][e]);
    }
    cur = next;
  }
#pragma unroll
  for (int m = 0; m < NT; ++m) red[warp][m][lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      float4 tot = red[0][m][lane];
#pragma unroll
      for (int y = 1; y < QD_WARPS; ++y) {
        const float4 v = red[y][m][lane];
        tot.x += v.x;
        tot.y += v.y;
        tot.z += v.z;
        tot.w += v.w;
      }
      q4_epilogue<NT>(a, tot, pre, m, n0, g, t);
    }
  }
}

// How a product is spread over the machine: the k range of a block (the
// cluster split), the warps that share a tile and the depth of the rings.
struct Q4Plan {
  int split, kr, ks, ring, part, grid;
  size_t smem;
};
bool q4_plan(int rows, int N, int K, int group, Q4Plan* p) {
  const int NR = rows <= 8 ? 8 : 16;
  const int slot = q4_slot(group);
  const int nst = (K + Q4_STAGE - 1) / Q4_STAGE, ntiles = (N + Q4_COLS - 1) / Q4_COLS;
  for (p->split = 1; p->split <= Q4_MAX_SPLIT; p->split *= 2) {
    p->kr = p->split == 1 ? K : (nst + p->split - 1) / p->split * Q4_STAGE;
    p->part = p->split > 1 ? Q4_PART_TILES : 0;
    if (p->split > 1 && q4_smem(NR, rows, p->kr, group, p->part).ring + 256 + 2 * Q4_WARPS * slot > Q4_SMEM) p->part = 1;
    const size_t fixed = q4_smem(NR, rows, p->kr, group, p->part).ring + 256;  // (256: the kernel's static words)
    if (fixed + (size_t)Q4_WARPS * 2 * slot > Q4_SMEM) continue;
    const int ring = (int)((Q4_SMEM - fixed) / ((size_t)Q4_WARPS * slot));
    p->ring = ring < 4 ? ring : 4;
    p->smem = fixed - 256 + (size_t)Q4_WARPS * p->ring * slot;
    break;
  }
  if (p->split > Q4_MAX_SPLIT) return false;
  const int slots = num_sms() / p->split;
  long best = -1;
  const int st = (p->kr + Q4_STAGE - 1) / Q4_STAGE;
  for (int ks = 1; ks <= Q4_WARPS; ks *= 2) {
    const int gpb = Q4_WARPS / ks;
    if (p->split > 1 && gpb > p->part) continue;
    const int per_block = (ntiles + slots - 1) / slots, passes = (per_block + gpb - 1) / gpb;
    const long cost = (long)passes * (2 * ((st + ks - 1) / ks) + 2);
    if (best < 0 || cost < best) {
      best = cost;
      p->ks = ks;
    }
  }
  p->grid = (ntiles < slots ? ntiles : slots) * p->split;
  return true;
}

template <int NT, int G>
int q4_launch(Q4Args& a, const Q4Plan& p, cudaStream_t st) {
  CUDA_TRY(once_per_device((const void*)q4_gemv_kernel<NT, G>, [](int) {
    return cudaFuncSetAttribute(q4_gemv_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q4_SMEM - 256);
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

template <int NT, int G, bool STAGED>
int q4_direct_launch(const Q4Args& a, cudaStream_t st) {
  const size_t smem = STAGED ? (size_t)a.rows * (a.K + QD_PAD) * sizeof(bf16) : 0;
  CUDA_TRY(once_per_device((const void*)q4_direct_kernel<NT, G, STAGED>, [](int) {
    return cudaFuncSetAttribute(q4_direct_kernel<NT, G, STAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                16 * (QD_STAGED_K + QD_PAD) * (int)sizeof(bf16));
  }));
  CUDA_TRY(launch_k(q4_direct_kernel<NT, G, STAGED>, (unsigned)((a.N + Q4_COLS - 1) / Q4_COLS), QD_WARPS * 32, smem, st, a));
  LAUNCH_CHECK();
  return GPT2_OK;
}
template <int NT, bool STAGED>
int q4_direct(const Q4Args& a, int group, cudaStream_t st) {
  if (group == 32) return q4_direct_launch<NT, 32, STAGED>(a, st);
  if (group == 64) return q4_direct_launch<NT, 64, STAGED>(a, st);
  return q4_direct_launch<NT, 128, STAGED>(a, st);
}

int q4_launch_rows(Q4Args& a, const Q4Plan& p, int group, cudaStream_t st) {
  a.ks = p.ks; a.split = p.split; a.kr = p.kr; a.ring = p.ring; a.part = p.part;
  int rows2 = 1;
  while (rows2 < a.rows) rows2 *= 2;
  a.wpr = Q4_WARPS / rows2;
  if (a.rows <= 8) {
    if (group == 32) return q4_launch<1, 32>(a, p, st);
    if (group == 64) return q4_launch<1, 64>(a, p, st);
    return q4_launch<1, 128>(a, p, st);
  }
  if (group == 32) return q4_launch<2, 32>(a, p, st);
  if (group == 64) return q4_launch<2, 64>(a, p, st);
  return q4_launch<2, 128>(a, p, st);
}

// Direct or streamed?  The direct kernel's time goes with its waves of blocks
// (two blocks an SM for up to 8 rows, but one in groups of 128 that are not
// staged) times the rounds in which a block's 16 warps walk the inputs; the
// streamed one's, from 5 us up, with the rows x inputs that it stages.
// Measured on both sides, in us (direct, streamed), 8 rows:
//   4736 x 768, groups of 32 (1 wave of 1 round) 3.3, 5.3; 9472 x 768 (2 of 1) 5.6, 5.6;
//   18944 x 128 (4 of 1) 7.8, 4.9; groups of 64, 4800 x 1664 (2 of 2) 5.4, 6.3;
//   1600 x 8192 (1 of 8, 65536 staged) 9.0, 11.8; 16 rows, 1600 x 12288 12.6, 24;
//   groups of 32, 1 row, 1600 x 6400 (1 of 7) 10.0, 7.5; 16 rows, 160 x 28672 34, 11.8.
// Over 435 sizes the choice is 2.1 % above the better one on average, at most
// 1.8 times (16 rows, 160 x 16384 in groups of 32).  Rows that are staged
// first pay in one wave: decode step of the 350M model, batch 1, with its QKV
// and fc products (1 wave) direct 559, streamed 602; batch 16 (2 waves of QKV)
// 997, 949; of the 1558M model, batch 1 (QKV: 2 waves) 1892, 1576.
bool q4_direct_pays(int rows, int N, int K, int group, bool staged) {
  const long tiles = (N + Q4_COLS - 1) / Q4_COLS, at_once = (long)num_sms() * (rows <= 8 && (staged || group < 128) ? 2 : 1);
  const long waves = (tiles + at_once - 1) / at_once, unit = QD_WARPS * (group < 64 ? 64 : group);
  const long rounds = (K + unit - 1) / unit;
  if (staged) return waves == 1 && K <= QD_STAGED_K;
  return (waves <= 2 && waves * rounds <= 4) || (waves == 1 && K <= 16384 && (long)rows * K >= 49152);
}

int q4_run(Q4Args& a, int group, cudaStream_t st) {
  if (q4_direct_pays(a.rows, a.N, a.K, group, a.ln || a.in_f32)) {
    if (!a.ln && !a.in_f32) return a.rows <= 8 ? q4_direct<1, false>(a, group, st) : q4_direct<2, false>(a, group, st);
    return a.rows <= 8 ? q4_direct<1, true>(a, group, st) : q4_direct<2, true>(a, group, st);
  }
  Q4Plan p;
  if (!q4_plan(a.rows, a.N, a.K, group, &p)) return GPT2_ERR_UNSUPPORTED_SHAPE;
  return q4_launch_rows(a, p, group, st);
}

// (K: at most 65535 k blocks of a grid; N: the ends of tiles stay inside 32 bits)
bool q4_shape_ok(int N, int K, int group) {
  return K <= 65535 * QZ_K && (group == 32 || group == 64 || group == 128) && N >= 0 && N <= 1 << 30 && K >= 1 && K % group == 0;
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
  if (N < 0 || K < 0 || ldw < K || (N && (!w || !packed || !scales))) return GPT2_ERR_INVALID_ARG;
  if (((uintptr_t)w | (uintptr_t)packed | (uintptr_t)scales) & 15) return GPT2_ERR_INVALID_ARG;
  if (!q4_shape_ok(N, K, group) || ldw % 8) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return GPT2_OK;
  return q4_quantize(w, w_fp32, ldw, N, K, group, packed, scales, reinterpret_cast<cudaStream_t>(stream));
}

int gpt2_op_q4_dequantize(const uint8_t* packed, const uint16_t* scales, int N, int K, int group, void* out,
                          int out_fp32, int ldo, void* stream) {
  if (N < 0 || K < 0 || ldo < K || (N && (!packed || !scales || !out))) return GPT2_ERR_INVALID_ARG;
  if (((uintptr_t)packed | (uintptr_t)scales | (uintptr_t)out) & 15) return GPT2_ERR_INVALID_ARG;
  if (!q4_shape_ok(N, K, group) || ldo % 8) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return GPT2_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long pitch = q4_pitch(N);
  const int shift = group == 32 ? 5 : (group == 64 ? 6 : 7);
  const bf16* sc = reinterpret_cast<const bf16*>(scales);
  const dim3 grid((N + 8 * DQ_ROWS - 1) / (8 * DQ_ROWS), (K + 255) / 256);
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
  if (rows < 0 || rows > 16 || N < 0 || K < 0 || ldx < K || ldo < N) return GPT2_ERR_INVALID_ARG;
  if (rows && N && (!x || !packed || !scales || !out)) return GPT2_ERR_INVALID_ARG;
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
