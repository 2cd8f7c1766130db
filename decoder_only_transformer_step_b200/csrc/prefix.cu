// Attention of one new token per sequence over a prefix that the whole batch
// shares and each sequence's own cached positions behind it.
//
//   z[j] = q . k[j] / sqrt(hd),  j over the P prefix keys and the row's own
//   o = sum_j exp(z[j] - lse) v[j],  lse = log sum_j exp(z[j])
//
// The query rows of a key/value head (batch x heads that share it) are the rows
// of one matrix product per block of keys, instead of B passes over the same
// keys: the prefix is read once for every 16 of them, or for up to 256 on
// tcgen05; only where it is short does each sequence read it for itself.  Work is split along the
// keys into parts of a fixed length; a part leaves, per row, its running
// maximum, sum and weighted values (fp32), and a second kernel joins a row's
// parts in a fixed order.  Rows without any key get o = 0, lse = -inf.
#include "attention_tc.cuh"
#include "common.cuh"
#include "internal.h"

namespace {

constexpr int PA_WARPS = 4;      // warps of a block: they share its part's keys
constexpr int PA_STAGES = 2;     // steps in a warp's ring
constexpr int PA_ROWS = 16;      // query rows of a block (the mma M)
constexpr int PA_BLOCKS = 444;   // blocks a call is spread over: 3 for each of 148 SMs
template <int HD> constexpr int pa_keys() { return HD == 128 ? 16 : 32; }  // keys of a warp's step
constexpr int PA_MIN_PART = PA_WARPS * 32;
// A block takes all keys of its rows, instead of parts that are joined, up to
// so many keys a row (the longer a key, the fewer) and so many bytes that the
// whole batch reads that way.  Measured on both sides, in us (all keys, parts),
// keys of 64: 16 rows, 12 heads, 256 keys (12.6 MB) 5.4, 7.0, 512 keys (25 MB)
// 7.15, 7.11, 768 keys 8.9, 7.6; 1 row, 12 heads, 512 keys 5.1, 5.5, 768 keys 6.1, 5.5;
// 40 rows, 25 heads, 200 keys (51 MB) 10.6, 12.1, 256 keys (66 MB) 12.4, 11.8.
// Keys of 128: 16 rows, 12 heads, 256 keys 8.0, 9.2, 384 keys 9.9, 9.6.  Keys of 16: 16 rows,
// 25 heads, 512 keys 5.8, 6.5, 640 keys 6.3, 6.2.
constexpr int pa_direct_keys(int hd) { return hd == 128 ? 256 : hd == 64 ? 512 : 640; }
constexpr double PA_DIRECT_BYTES = 55e6;
constexpr int PT_BLOCKS = 148;   // blocks of the tcgen05 kernel: one an SM
// The tcgen05 kernel is taken from so many query rows of a key/value head on,
// where their products with the prefix are so many (rows x keys x hd).
// Measured on both sides, in us (tcgen05, mma.sync): 48 rows, 16384 keys of 128,
// 8 heads (1.0e8) 27.5, 28.6; 128 rows, 16384 keys of 64, 12 heads (1.3e8) 39, 47;
// 128 rows, 3500 keys of 128 (5.7e7) 26.3, 26.7; 64 rows, 16384 keys of 64 (6.7e7)
// 31, 27; 32 rows, 16384 keys of 128 26.4, 24.0.
constexpr int PT_MIN_ROWS = 48;
constexpr double PT_MIN_WORK = 9e7;

struct PrefixArgs {
  const void* q;  // [B, ldq], bf16 or fp32 (rounded to bf16 on load)
  long ldq;
  int q_aligned;  // rows of q at 16-byte boundaries
  const bf16 *pk, *pv;  // [Hkv][pcap][hd]
  int P;
  long pcap;
  const bf16 *k, *v;  // [B][Hkv][max_len][hd]
  const int32_t* len;
  int len_add, max_len;
  int B, Hq, Hkv, G;
  float scale_log2;
  int Lp, Lo;         // keys of a part of the prefix / of a row's own keys
  int nsp, nso;       // parts of the prefix, parts of a row's own keys (at most)
  int direct;         // a block takes all keys of its rows
  int tc;             // the prefix's parts are prefix_tc_kernel's
  int mtp, mto;       // 16-row tiles of a key/value head's rows in the prefix / of its group
  float* po;          // [nsp + nso][B * Hq][hd]
  float2* pml;        // [nsp + nso][B * Hq]: maximum (log2 units), sum
};

DEVI int own_len(const PrefixArgs& a, int b) {
  if (a.max_len == 0) return 0;  // len may be NULL
  const int n = a.len[b] + a.len_add;
  return n < 0 ? 0 : (n > a.max_len ? a.max_len : n);
}

DEVI void cp_async16z(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // 0: the 16 bytes are zeroed, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
DEVI void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
DEVI void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
DEVI void pa_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename QT> DEVI uint32_t ld_q2(const QT* p);
template <> DEVI uint32_t ld_q2<bf16>(const bf16* p) { return *reinterpret_cast<const uint32_t*>(p); }
template <> DEVI uint32_t ld_q2<float>(const float* p) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  return pack_bf16x2(v.x, v.y);
}

template <int HD> constexpr int pa_smem() {
  constexpr int ring = PA_WARPS * PA_STAGES * 2 * pa_keys<HD>() * HD * 2, join = PA_WARPS * PA_ROWS * ((HD + 4) * 4 + 8);
  return ring > join ? ring : join;
}

// One part of the keys for up to 16 query rows.  Bound by HBM reads of keys
// and values: 4 hd bytes a key feed 16 rows' products (mma.sync m16n8k16),
// which take a few percent of the tensor cores' time, so each warp streams
// its own steps of 16 or 32 keys through a ring of its own (cp.async, a step
// ahead) without block-wide waits, with its own running maximum and sum; the
// warps meet once at the end.  Probabilities are rounded to bf16 for the
// second product (its operand type; their sum stays fp32 of the unrounded
// ones): half a step, 2^-8 relative at most, as the output's own rounding, and
// 1.1 times the error of a bf16 output of unrounded ones.  (A second product
// with what the rounding leaves costs 6 to 15 %: 16 x 12 x 3500 9.7 -> 10.3 us, 1 x
// 12 x 400 5.0 -> 5.8.)
// Where a row has few keys in all and the whole batch reads little (DIRECT), a
// block takes all keys of its rows instead, those of the prefix and then their
// own, and writes the output itself: 3 rows, 12 heads, 200 + 64 keys of 64 in
// 4.2 us (5.2 in parts and joined).  In parts, 16 rows, 12 heads, 3500 + 596 keys
// take 9.8 us with the join, bound by the two kernels' waits for memory (28 % of
// HBM, issue slots 28 % busy).
template <int HD, typename QT, bool DIRECT>
__global__ void __launch_bounds__(PA_WARPS * 32)
    prefix_part_kernel(const __grid_constant__ PrefixArgs a, bf16* __restrict__ out, long ldo, float* __restrict__ lse) {
  extern __shared__ __align__(128) uint8_t pa_smem_buf[];
  constexpr int PA_KEYS = pa_keys<HD>();
  constexpr int C = HD / 8;                       // 16-byte chunks of a key
  constexpr int SWZ = C < 8 ? C - 1 : 7;          // chunk index ^ (key & SWZ): ldmatrix rows in distinct banks
  constexpr int KB = PA_KEYS * HD * 2;            // bytes of a step's keys (and of its values)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_trigger();
  pdl_wait();
  // which part: those of the prefix first (the tiles of one key range next to
  // each other, for L2), then the rows' own
  const int np = DIRECT || a.tc ? 0 : a.nsp * a.Hkv * a.mtp;
  int x = blockIdx.x, part, h, mt, b0 = 0, n, nrows;
  const bf16 *kb, *vb;
  const bool shared_keys = x < np;
  if (shared_keys) {
    mt = x % a.mtp;
    h = x / a.mtp % a.Hkv;
    part = x / (a.mtp * a.Hkv);
    n = a.P;
    kb = a.pk + (size_t)h * a.pcap * HD;
    vb = a.pv + (size_t)h * a.pcap * HD;
    nrows = a.B * a.G;
  } else {
    x -= np;
    mt = x % a.mto;
    h = x / a.mto % a.Hkv;
    b0 = x / (a.mto * a.Hkv) % a.B;
    part = x / (a.mto * a.Hkv * a.B);
    n = own_len(a, b0);
    kb = a.k + ((size_t)b0 * a.Hkv + h) * a.max_len * HD;
    vb = a.v + ((size_t)b0 * a.Hkv + h) * a.max_len * HD;
    nrows = a.G;
  }
  const int L = shared_keys ? a.Lp : a.Lo;
  const int k0 = DIRECT ? 0 : part * L, k1 = DIRECT ? n : min(n, k0 + L);
  if (!DIRECT && k0 >= k1) return;
  // row i of the tile -> (sequence, query head)
  auto row_of = [&](int i, int* b, int* hq) {
    const int m = mt * PA_ROWS + i;
    *b = shared_keys ? m / a.G : b0;
    *hq = h * a.G + (shared_keys ? m % a.G : m);
    return m < nrows;
  };
  const uint32_t ring = smem_u32(pa_smem_buf) + warp * (PA_STAGES * 2 * KB);
  const int psteps = DIRECT ? (a.P + PA_KEYS - 1) / PA_KEYS : 0;  // (DIRECT) steps of the prefix, before the row's own
  const int nsteps = psteps + (k1 - k0 + PA_KEYS - 1) / PA_KEYS;
  int ps = warp, pslot = 0;
  auto issue = [&]() {
    if (ps < nsteps) {
      const bool pre = DIRECT && ps < psteps;
      const int j0 = pre ? ps * PA_KEYS : k0 + (ps - psteps) * PA_KEYS, end = pre ? a.P : k1;
      const bf16* ks = pre ? a.pk + (size_t)h * a.pcap * HD : kb;
      const bf16* vs = pre ? a.pv + (size_t)h * a.pcap * HD : vb;
      const uint32_t dst = ring + pslot * 2 * KB;
#pragma unroll
      for (int i = 0; i < PA_KEYS * C / 32; ++i) {
        const int e = lane + 32 * i, key = e / C, ch = e % C;
        const bool live = j0 + key < end;
        const size_t at = (size_t)(live ? j0 + key : j0) * HD + ch * 8;
        const uint32_t d = dst + key * (HD * 2) + ((ch ^ (key & SWZ)) << 4);
        cp_async16z(d, ks + at, live);
        cp_async16z(d + KB, vs + at, live);
      }
      ps += PA_WARPS;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    pslot = pslot + 1 == PA_STAGES ? 0 : pslot + 1;
  };
#pragma unroll
  for (int i = 0; i < PA_STAGES - 1; ++i) issue();

  uint32_t qf[HD / 16][4];
  {
    int ba, ha, bb, hb;
    const bool la = row_of(g, &ba, &ha), lb = row_of(g + 8, &bb, &hb);
    const QT* qa = reinterpret_cast<const QT*>(a.q) + (la ? (size_t)ba * a.ldq + ha * HD : 0) + 2 * t;
    const QT* qb = reinterpret_cast<const QT*>(a.q) + (lb ? (size_t)bb * a.ldq + hb * HD : 0) + 2 * t;
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) {
      qf[c][0] = la ? ld_q2<QT>(qa + 16 * c) : 0u;
      qf[c][1] = lb ? ld_q2<QT>(qb + 16 * c) : 0u;
      qf[c][2] = la ? ld_q2<QT>(qa + 16 * c + 8) : 0u;
      qf[c][3] = lb ? ld_q2<QT>(qb + 16 * c + 8) : 0u;
    }
  }
  // running maximum (in log2 units of the scaled scores), sum, values
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, o[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  // ldmatrix addresses: K as 8x8 (keys, dims) tiles, V transposed
  const int kkey = ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;
  const int vkey = (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;
  int cslot = 0;
  for (int s = warp; s < nsteps; s += PA_WARPS) {
    asm volatile("cp.async.wait_group %0;" ::"n"(PA_STAGES - 2) : "memory");
    __syncwarp();
    issue();
    const uint32_t kt = ring + cslot * 2 * KB, vt = kt + KB;
    float z[PA_KEYS / 8][4];
#pragma unroll
    for (int i = 0; i < PA_KEYS / 8; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) {
#pragma unroll
      for (int j = 0; j < PA_KEYS / 16; ++j) {
        uint32_t r[4];
        const int key = 16 * j + kkey;
        ldsm4(kt + key * (HD * 2) + (((2 * c + kch) ^ (key & SWZ)) << 4), r);
        pa_mma(z[2 * j], qf[c], r[0], r[1]);
        pa_mma(z[2 * j + 1], qf[c], r[2], r[3]);
      }
    }
    const int left = DIRECT && s < psteps ? a.P - s * PA_KEYS : k1 - (k0 + (s - psteps) * PA_KEYS);
    if (left < PA_KEYS) {
#pragma unroll
      for (int i = 0; i < PA_KEYS / 8; ++i) {
        const int key = 8 * i + 2 * t;
        if (key >= left) z[i][0] = z[i][2] = -INFINITY;
        if (key + 1 >= left) z[i][1] = z[i][3] = -INFINITY;
      }
    }
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < PA_KEYS / 8; ++i) {
      x0 = fmaxf(x0, fmaxf(z[i][0], z[i][1]));
      x1 = fmaxf(x1, fmaxf(z[i][2], z[i][3]));
    }
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
    x0 *= a.scale_log2;
    x1 *= a.scale_log2;
    if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
      const float y0 = fmaxf(m0, x0), y1 = fmaxf(m1, x1);
      const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - y0), f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - y1);
      m0 = y0;
      m1 = y1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f0;
        o[i][2] *= f1;
        o[i][3] *= f1;
      }
    }
    const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
    for (int i = 0; i < PA_KEYS / 8; ++i) {
      z[i][0] = ex2_approx(fmaf(z[i][0], a.scale_log2, -r0));
      z[i][1] = ex2_approx(fmaf(z[i][1], a.scale_log2, -r0));
      z[i][2] = ex2_approx(fmaf(z[i][2], a.scale_log2, -r1));
      z[i][3] = ex2_approx(fmaf(z[i][3], a.scale_log2, -r1));
      l0 += z[i][0] + z[i][1];
      l1 += z[i][2] + z[i][3];
    }
#pragma unroll
    for (int j = 0; j < PA_KEYS / 16; ++j) {
      const uint32_t p[4] = {pack_bf16x2(z[2 * j][0], z[2 * j][1]), pack_bf16x2(z[2 * j][2], z[2 * j][3]),
                             pack_bf16x2(z[2 * j + 1][0], z[2 * j + 1][1]), pack_bf16x2(z[2 * j + 1][2], z[2 * j + 1][3])};
      const int key = 16 * j + vkey;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        uint32_t r[4];
        ldsm4t(vt + key * (HD * 2) + (((2 * c + vch) ^ (key & SWZ)) << 4), r);
        pa_mma(o[2 * c], p, r[0], r[1]);
        pa_mma(o[2 * c + 1], p, r[2], r[3]);
      }
    }
    cslot = cslot + 1 == PA_STAGES ? 0 : cslot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  // the warps' sums meet in shared memory (over the rings, all of whose
  // copies have landed): [warp][16][HD + 4] values, [warp][16] (maximum, sum)
  __syncthreads();
  constexpr int OP = HD + 4;
  float* so = reinterpret_cast<float*>(pa_smem_buf);
  float2* sml = reinterpret_cast<float2*>(so + PA_WARPS * PA_ROWS * OP);
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) {
    float* d = so + (warp * PA_ROWS + g) * OP + 8 * i + 2 * t;
    *reinterpret_cast<float2*>(d) = make_float2(o[i][0], o[i][1]);
    *reinterpret_cast<float2*>(d + 8 * OP) = make_float2(o[i][2], o[i][3]);
  }
  if (t == 0) {
    sml[warp * PA_ROWS + g] = make_float2(m0, l0);
    sml[warp * PA_ROWS + g + 8] = make_float2(m1, l1);
  }
  __syncthreads();
  const int slot = shared_keys ? part : a.nsp + part;
  for (int i = threadIdx.x; i < PA_ROWS * (HD / 4); i += PA_WARPS * 32) {
    const int row = i / (HD / 4), c = i % (HD / 4) * 4;
    int b, hq;
    if (!row_of(row, &b, &hq)) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < PA_WARPS; ++w) M = fmaxf(M, sml[w * PA_ROWS + row].x);
    float lsum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < PA_WARPS; ++w) {
      const float2 ml = sml[w * PA_ROWS + row];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      const float4 ow = *reinterpret_cast<const float4*>(so + (w * PA_ROWS + row) * OP + c);
      lsum = fmaf(f, ml.y, lsum);
      v.x = fmaf(f, ow.x, v.x);
      v.y = fmaf(f, ow.y, v.y);
      v.z = fmaf(f, ow.z, v.z);
      v.w = fmaf(f, ow.w, v.w);
    }
    if constexpr (DIRECT) {
      const bool any = nsteps > 0;
      const float inv = any ? 1.f / lsum : 0.f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(out + (size_t)b * ldo + (size_t)hq * HD + c);  // (4-byte aligned)
      dst[0] = pack_bf16x2(v.x * inv, v.y * inv);
      dst[1] = pack_bf16x2(v.z * inv, v.w * inv);
      if (lse && c == 0) lse[(size_t)b * a.Hq + hq] = any ? fmaf(M, 0.6931471805599453f, logf(lsum)) : -INFINITY;
    } else {
      const size_t at = (size_t)slot * a.B * a.Hq + (size_t)b * a.Hq + hq;
      *reinterpret_cast<float4*>(a.po + at * HD + c) = v;
      if (c == 0) a.pml[at] = make_float2(M, lsum);
    }
  }
}

// ------------------------------------------------- many rows: tcgen05 ------
// The prefix's parts where a key/value head has many query rows: the products
// S = Q K^T (M 128, N 64) and O += P V on the 5th-generation tensor cores, so
// that up to 256 rows share one pass over the keys.  One block per (key range,
// key/value head, row group):
//   warp 0        TMA: K and V tiles of 128 keys, alternately, through a ring
//   warps 1, 2    MMA issue of row tile 0 / 1 (warp 1 also owns the TMEM)
//   warps 4..7    softmax of tile 0, warps 8..11 of tile 1, a thread a row
// A step is 64 keys.  Tensor memory of a tile: two buffers of S (64 fp32
// columns), over which the step's bf16 probabilities P (32 columns) are
// written once S has been read, and O (hd).  S of the next step is issued
// before P V of this one, so that the softmax waits little for the tensor cores
// (200 to 420 cycles a step).  A row rescales its O only when its maximum grows by more than 2^8 (the
// probabilities are formed against the older maximum, exact in the final O /
// l).  Warps without rows take no part.  160 rows over 32768 keys of 128, 8
// heads: 46 us (37 % of HBM, tensor pipe 43 %), about 1950 cycles a step, of
// which two softmax warps that share a scheduler take 1600 to 1690, one alone 950:
// bound by their instructions (a quarter of the exponentials on the FMA pipe
// instead: a call 57.6 -> 59.2 us).
// Every wait is bounded; after one that ran out the part's rows become NaN.
constexpr float PT_RESCALE = 8.f;
template <int HD> constexpr int pt_slots() { return HD == 128 ? 5 : 8; }
template <int HD> constexpr int pt_tile() { return 128 * HD * 2; }  // bytes of a 128-row tile
template <int HD, int NT> constexpr int pt_tiles() { return (NT + pt_slots<HD>()) * pt_tile<HD>(); }
template <int HD, int NT> constexpr int pt_bars() { return 2 * pt_slots<HD>() + 7 * NT; }
template <int HD, int NT> constexpr int pt_smem() { return pt_tiles<HD, NT>() + 1024 + pt_bars<HD, NT>() * 8 + 16; }
// S: M 128, N 64, both K-major; P V: M 128, N hd, V MN-major (its 64-column halves 16 KB apart)
constexpr uint32_t PT_IDESC_S = (1u << 4) | (1u << 7) | (1u << 10) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t pt_idesc_o(int hd) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (((uint32_t)hd >> 3) << 17) | ((128u >> 4) << 24);
}
constexpr int PT_REGS_CTRL = 80, PT_REGS_SOFT = 208;
static_assert(128 * PT_REGS_CTRL + 256 * PT_REGS_SOFT <= 384 * 168, "register split");

// Rows of tile t of a group of n: whole warps, the first tile the larger half.
__host__ __device__ inline int pt_rows(int n, int nt, int t) {
  if (nt == 1) return n;
  const int r0 = min((n + 1) / 2 + 31, n + 31) / 32 * 32;
  return t == 0 ? min(r0, n) : n - min(r0, n);
}

template <int HD, int NT>
__global__ void __launch_bounds__(128 + 128 * NT, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PrefixArgs a) {
  constexpr int NS = pt_slots<HD>(), TB = pt_tile<HD>(), SUB = 128 * 128;  // SUB: 128 rows x 64 columns, 128B-swizzled
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t bars = base + pt_tiles<HD, NT>();
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + pt_tiles<HD, NT>() + pt_bars<HD, NT>() * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto kv_full = [&](int s) { return bars + 8u * s; };
  auto kv_empty = [&](int s) { return bars + 8u * (NS + s); };
  // per tile: 0 q_full, 1 2 s_full, 3 4 p_full (of even and odd steps), 5 pv_done, 6 drain
  auto tbar = [&](int t, int k) { return bars + 8u * (2 * NS + 7 * t + k); };
  auto q_tile = [&](int t) { return base + (uint32_t)(t * TB); };
  auto kv_tile = [&](int s) { return base + (uint32_t)((NT + s) * TB); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (row group fastest: the blocks of one key range next to each other, for L2)
  const int mg = blockIdx.x % a.mtp, h = blockIdx.x / a.mtp % a.Hkv, part = blockIdx.x / (a.mtp * a.Hkv);
  const int k0 = part * a.Lp, k1 = min(a.P, k0 + a.Lp), nh = (k1 - k0 + 63) / 64, nb = (nh + 1) / 2;
  const int M = a.B * a.G, per = (M + a.mtp - 1) / a.mtp, m0 = mg * per, mrows = min(per, M - m0);  // this group's rows
  auto rows_of = [&](int t) { return pt_rows(mrows, NT, t); };

  if (threadIdx.x == 0) {
    int tiles = 0;
    for (int t = 0; t < NT; ++t) tiles += rows_of(t) > 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), tiles);
    }
    for (int t = 0; t < NT; ++t) {
      const int warps = max(1, (rows_of(t) + 31) / 32);
      mbar_init(tbar(t, 0), warps);
      mbar_init(tbar(t, 1), 1);
      mbar_init(tbar(t, 2), 1);
      mbar_init(tbar(t, 3), warps);
      mbar_init(tbar(t, 4), warps);
      mbar_init(tbar(t, 5), 1);
      mbar_init(tbar(t, 6), 1);
    }
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 256 * NT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_start();

  if (warp < 4) {
    if constexpr (NT == 2) reg_dealloc<PT_REGS_CTRL>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------- TMA ----
      // tile 2 j is K of block j, tile 2 j + 1 its V
      int issued = 0;
      for (int i = 0; i < 2 * nb; ++i) {
        const int s = i % NS;
        if (i >= NS && !mbar_wait_bounded(kv_empty(s), ((i - NS) / NS) & 1, abort_flag, nullptr)) break;
        mbar_arrive_expect_tx(kv_full(s), TB);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
          tma_load_3d(kv_tile(s) + c * SUB, (i & 1) ? &tmV : &tmK, kv_full(s), 64 * c, k0 + (i >> 1) * 128, h);
        ++issued;
      }
      // (all have landed, unless the others gave up: no copy may arrive after the block has left)
      for (int i = issued - NS < 0 ? 0 : issued - NS; i < issued; ++i) mbar_drain_bounded(kv_full(i % NS), (i / NS) & 1);
    } else if ((warp == 1 || (NT == 2 && warp == 2)) && lane == 0 && rows_of(warp - 1) > 0) {
      // ------------------------------------------------------------- MMA ----
      const int t = warp - 1;
      const uint32_t tS = tmem + 256u * t, tO = tS + 128u;
      bool ok = mbar_wait_bounded(tbar(t, 0), 0, abort_flag, nullptr), issued = false;
      auto issue_s = [&](int i) -> bool {
        const int kt = i & ~1, s = kt % NS;  // (tile 2 j of block j = i / 2)
        if (!(i & 1) && !mbar_wait_bounded(kv_full(s), (kt / NS) & 1, abort_flag, nullptr)) return false;
        // P V of the step before last has read the P that this S goes over
        if (i >= 2 && !mbar_wait_bounded(tbar(t, 5), i & 1, abort_flag, nullptr)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = (k >> 2) * SUB + (k & 3) * 32;
          tc_mma_bf16(tS + 64u * (i & 1), sdesc(q_tile(t) + off, 16, 1024),
                      sdesc(kv_tile(s) + off + (i & 1) * 8192, 16, 1024), PT_IDESC_S, k > 0 ? 1u : 0u);
        }
        issued = true;
        tc_commit(tbar(t, 1 + (i & 1)));
        if ((i & 1) || i + 1 == nh) tc_commit(kv_empty(s));
        return true;
      };
      ok = ok && issue_s(0);
      for (int i = 0; i < nh && ok; ++i) {
        const int vt = i | 1, s = vt % NS;
        if ((i + 1 < nh && !issue_s(i + 1)) ||
            (!(i & 1) && !mbar_wait_bounded(kv_full(s), (vt / NS) & 1, abort_flag, nullptr)) ||
            !mbar_wait_bounded(tbar(t, 3 + (i & 1)), (i >> 1) & 1, abort_flag, nullptr)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_bf16_ts(tO, tS + 64u * (i & 1) + 8u * k, sdesc(kv_tile(s) + (4 * (i & 1) + k) * 2048, SUB, 1024),
                         pt_idesc_o(HD), (i > 0 || k > 0) ? 1u : 0u);
        tc_commit(tbar(t, 5));
        if ((i & 1) || i + 1 == nh) tc_commit(kv_empty(s));
      }
      if (issued) {  // (whoever gave up: none of this warp's products is in flight when the tensor memory is freed)
        tc_commit(tbar(t, 6));
        mbar_drain_bounded(tbar(t, 6), 0);
      }
    }
  } else {
    if constexpr (NT == 2) reg_alloc<PT_REGS_SOFT>();
    // ----------------------------------------------------------- softmax ----
    // The lanes of quarter q hold the tile's rows 32 q ..; in tile 1 the
    // quarters are taken from the other end, so that the warps of two partly
    // filled tiles share the schedulers evenly.
    const int t = (warp - 4) >> 2, q = warp & 3, at = q * 32 + lane, lr = (t ? 3 - q : q) * 32 + lane;
    const int rows = rows_of(t);
    if ((lr & ~31) < rows) {
      const bool live = lr < rows;
      const int m = m0 + (t ? rows_of(0) : 0) + (live ? lr : 0), b = m / a.G, hq = h * a.G + m % a.G;
      {
        // this thread's row of Q, K-major and 128-byte swizzled
        const bf16* src = reinterpret_cast<const bf16*>(a.q) + (size_t)b * a.ldq + (size_t)hq * HD;
        const uint32_t row = q_tile(t) + (uint32_t)at * 128u;
        uint32_t w[HD / 8][4];
        if (a.q_aligned) {
#pragma unroll
          for (int c = 0; c < HD / 8; ++c) {
            const uint4 u = *reinterpret_cast<const uint4*>(src + 8 * c);
            w[c][0] = u.x; w[c][1] = u.y; w[c][2] = u.z; w[c][3] = u.w;
          }
        } else {
#pragma unroll
          for (int c = 0; c < HD / 8; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[c][e] = ld_q2<bf16>(src + 8 * c + 2 * e);
        }
        // (the lanes without a row hold the group's first: finite, and dropped)
#pragma unroll
        for (int c = 0; c < HD / 8; ++c)
          st_shared_v4(row + (c >> 3) * SUB + 16u * (uint32_t)((c & 7) ^ (at & 7)), w[c][0], w[c][1], w[c][2], w[c][3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(tbar(t, 0));
      }
      const uint32_t tS = tmem + ((uint32_t)(q * 32) << 16) + 256u * t, tO = tS + 128u;
      const float scale = a.scale_log2;
      float m_use = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = 0; i < nh; ++i) {
        const uint32_t tSi = tS + 64u * (i & 1);
        if (!mbar_wait_bounded(tbar(t, 1 + (i & 1)), (i >> 1) & 1, abort_flag, nullptr)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x32(tSi + 32u * c, v[c]);
        tmem_ld_wait();
        const int left = k1 - (k0 + 64 * i);  // keys of this step and behind it
        if (left < 64) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= left) v[c][e] = 0xff800000u;
        }
        float mxs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mxs[e] = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mxs[(e >> 1) & 7] = fmax3(mxs[(e >> 1) & 7], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
        const float mx = fmaxf(fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])),
                               fmaxf(fmaxf(mxs[4], mxs[5]), fmaxf(mxs[6], mxs[7])));
        const float m_new = fmaxf(m_use, mx * scale);
        float alpha = 1.f;
        bool rescale = false;
        if (i == 0) {
          m_use = m_new;
        } else if (m_new > m_use + PT_RESCALE) {
          alpha = ex2_approx(m_use - m_new);
          m_use = m_new;
          rescale = true;
        }
        const float ref = m_use == -INFINITY ? 0.f : m_use;  // (no finite score yet)
        float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(-ref, -ref);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), sc2, nm2);
            const float2 pr = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sums[e & 1] = __fadd2_rn(sums[e & 1], pr);
            pk[e] = pack_bf16x2(pr.x, pr.y);
          }
          // (all of this warp's S has been loaded: P goes over it)
          tmem_st_32x32b_x16(tSi + 16u * c, pk);
        }
        l = l * alpha + ((sums[0].x + sums[0].y) + (sums[1].x + sums[1].y));
        // rare: rows whose maximum grew rescale their O, once the P V before is in it
        if (__any_sync(0xffffffffu, rescale)) {
          if (!mbar_wait_bounded(tbar(t, 5), (i - 1) & 1, abort_flag, nullptr)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + 32u * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x32(tO + 32u * c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tbar(t, 3 + (i & 1)));
      }
      // (the last S implied P V of the step nh - 3; a phase is waited for only once the one before it is known complete)
      if (ok && nh >= 2) ok = mbar_wait_bounded(tbar(t, 5), (nh - 2) & 1, abort_flag, nullptr);
      if (ok) ok = mbar_wait_bounded(tbar(t, 5), (nh - 1) & 1, abort_flag, nullptr);
      tc_fence_after();
      const size_t slot = (size_t)part * a.B * a.Hq + (size_t)b * a.Hq + hq;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tO + 32u * c, o);
        tmem_ld_wait();
        if (live)
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(a.po + slot * HD + 32 * c + i) =
                make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
      }
      if (live) a.pml[slot] = ok ? make_float2(m_use, l) : make_float2(0.f, __int_as_float(0x7fffffff));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256 * NT);
  }
}

// Joins the parts of a row (in the order of the parts): a block a row, its
// warps take the parts in turn, a lane the same dims of each.  Bound by the
// waits for the parts: 6 us for 192 rows, 10 for 1280 of 128 dims (cold caches).
template <int HD>
__global__ void __launch_bounds__(128)
    prefix_join_kernel(const __grid_constant__ PrefixArgs a, bf16* __restrict__ o, long ldo, float* __restrict__ lse) {
  constexpr int V = HD >= 128 ? 4 : 2;   // dims of a lane
  constexpr int NL = HD / V;             // lanes at work (8 at hd 16)
  constexpr int U = 8;                   // parts in flight
  __shared__ float so[4][HD];
  __shared__ float2 sml[4];
  pdl_start();
  const int row = blockIdx.x, b = row / a.Hq, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nown = (own_len(a, b) + a.Lo - 1) / a.Lo, n = a.nsp + nown;  // the row's parts: slots 0 .. n - 1
  const size_t rows = (size_t)a.B * a.Hq;
  float M = -INFINITY, l = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int p0 = warp; p0 < n; p0 += 4 * U) {
    float2 ml[U];
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + 4 * u;
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) v[u][e] = 0.f;
      if (p < n) {
        const size_t at = (size_t)p * rows + row;
        ml[u] = a.pml[at];
        if (lane < NL) {
          const float* src = a.po + at * HD + lane * V;
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 w = *reinterpret_cast<const float2*>(src + e);
            v[u][e] = w.x;
            v[u][e + 1] = w.y;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + 4 * u >= n) break;
      const float Mn = fmaxf(M, ml[u].x);
      const float fa = M == -INFINITY ? 0.f : ex2_approx(M - Mn), fb = ml[u].x == -INFINITY ? 0.f : ex2_approx(ml[u].x - Mn);
      M = Mn;
      l = l * fa + ml[u].y * fb;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = acc[e] * fa + v[u][e] * fb;
    }
  }
  if (lane < NL)
#pragma unroll
    for (int e = 0; e < V; ++e) so[warp][lane * V + e] = acc[e];
  if (lane == 0) sml[warp] = make_float2(M, l);
  __syncthreads();
  float T = -INFINITY, L = 0.f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) T = fmaxf(T, sml[w].x);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = sml[w].x == -INFINITY ? 0.f : ex2_approx(sml[w].x - T);
    L = fmaf(f[w], sml[w].y, L);
  }
  const float inv = n > 0 ? 1.f / L : 0.f;
  if (threadIdx.x < HD / 2) {
    const int e = 2 * threadIdx.x;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      x = fmaf(f[w], so[w][e], x);
      y = fmaf(f[w], so[w][e + 1], y);
    }
    *reinterpret_cast<uint32_t*>(o + (size_t)b * ldo + (size_t)(row % a.Hq) * HD + e) = pack_bf16x2(x * inv, y * inv);
  }
  if (lse && threadIdx.x == 0) lse[row] = n > 0 ? fmaf(T, 0.6931471805599453f, logf(L)) : -INFINITY;
}

// The correctness mode's form, all fp32 on CUDA cores: one warp a (row, head),
// a lane HD / 32 dims (at hd 16 half the lanes), keys one by one.
template <int HD>
__global__ void __launch_bounds__(32)
    prefix_f32_kernel(const float* q, const float* pk, const float* pv, int P, long pcap, const float* k, const float* v,
                      const int32_t* len, int len_add, int max_len, int H, float scale, float* __restrict__ o) {
  constexpr int V = HD >= 32 ? HD / 32 : 1;
  pdl_start();
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x, d = H * HD;
  int n = len[b] + len_add;
  n = n < 0 ? 0 : (n > max_len ? max_len : n);
  float qv[V], acc[V], m = -INFINITY, l = 0.f;
  const bool live = lane * V < HD;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    qv[e] = live ? q[(size_t)b * d + h * HD + lane * V + e] * scale : 0.f;
    acc[e] = 0.f;
  }
  for (int j = 0; j < P + n; ++j) {
    const size_t at = j < P ? ((size_t)h * pcap + j) * HD : (((size_t)b * H + h) * max_len + (j - P)) * HD;
    const float *kr = (j < P ? pk : k) + at, *vr = (j < P ? pv : v) + at;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (live) s = fmaf(qv[e], kr[lane * V + e], s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), fa = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * fa + p;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (live) acc[e] = acc[e] * fa + p * vr[lane * V + e];
  }
  const float inv = P + n > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (live) o[(size_t)b * d + h * HD + lane * V + e] = acc[e] * inv;
}

// The split of a call, from the sizes alone, not the device: the scratch a
// caller sizes without one is the scratch a call uses.
struct PrefixPlan {
  int direct, tc, Lp, Lo, nsp, nso, mtp, mto;
  size_t rows, po_bytes, bytes;
};
bool prefix_plan(int B, int Hq, int Hkv, int hd, int P, int max_len, PrefixPlan* p) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || P < 0 || max_len < 0) return false;
  if (P > 1 << 30 || max_len > 1 << 30) return false;  // (the ends of parts stay inside 32 bits)
  if (hd != 16 && hd != 64 && hd != 128) return false;
  const int G = Hq / Hkv;
  const long M = (long)B * G;
  p->mto = (G + PA_ROWS - 1) / PA_ROWS;
  const long own_blocks = (long)B * Hkv * p->mto;
  // parts of at least `least` keys, a multiple of it, so that `blocks` blocks share `keys`
  auto part = [](double keys, long blocks, long least, long longest) {
    long L = (long)(keys / blocks) + 1;
    L = (L + least - 1) / least * least;
    if (L > longest + least) L = (longest + least) / least * least;
    return (int)L;
  };
  p->direct = (long)P + max_len <= pa_direct_keys(hd) &&
              (double)own_blocks * ((double)P + max_len) * hd * 4 <= PA_DIRECT_BYTES;
  p->tc = !p->direct && hd >= 64 && M >= PT_MIN_ROWS && (double)M * P * hd >= PT_MIN_WORK;
  if (p->tc) {
    const long max_rows = M <= 128 ? 128 : 256;
    p->mtp = (int)((M + max_rows - 1) / max_rows);
    long parts = PT_BLOCKS / ((long)Hkv * p->mtp);  // one block an SM
    if (parts < 1) parts = 1;
    p->Lp = part((double)P, parts, 128, P);
    p->Lo = part((double)own_blocks * max_len, PA_BLOCKS, PA_MIN_PART, max_len);
  } else {
    p->mtp = (int)((M + PA_ROWS - 1) / PA_ROWS);
    p->Lp = p->Lo = part((double)Hkv * p->mtp * P + (double)own_blocks * max_len, PA_BLOCKS, PA_MIN_PART,
                         P > max_len ? P : max_len);
  }
  p->nsp = (int)(((long)P + p->Lp - 1) / p->Lp);
  p->nso = (int)(((long)max_len + p->Lo - 1) / p->Lo);
  p->rows = (size_t)B * Hq;
  p->po_bytes = ((size_t)(p->nsp + p->nso) * p->rows * hd * 4 + 255) & ~(size_t)255;
  p->bytes = p->po_bytes + (((size_t)(p->nsp + p->nso) * p->rows * 8 + 255) & ~(size_t)255);
  if (p->bytes == 0) p->bytes = 256;
  return true;
}

template <int HD, int NT>
int prefix_tc_run(const PrefixArgs& a, cudaStream_t st) {
  CUtensorMap tk, tv;
  const uint64_t dims[3] = {HD, (uint64_t)a.P, (uint64_t)a.Hkv};
  const uint64_t strides[2] = {HD * 2, (uint64_t)a.pcap * HD * 2};
  if (!tmap_3d(&tk, a.pk, dims, strides) || !tmap_3d(&tv, a.pv, dims, strides)) return GPT2_ERR_CUDA;
  CUDA_TRY(once_per_device((const void*)prefix_tc_kernel<HD, NT>, [](int) {
    return cudaFuncSetAttribute(prefix_tc_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                pt_smem<HD, NT>());
  }));
  CUDA_TRY(launch_k(prefix_tc_kernel<HD, NT>, dim3((unsigned)(a.nsp * a.Hkv * a.mtp)), 128 + 128 * NT,
                    (size_t)pt_smem<HD, NT>(), st, tk, tv, a));
  LAUNCH_CHECK();
  return GPT2_OK;
}

template <int HD, typename QT>
int prefix_run(const PrefixArgs& a, bf16* o, long ldo, float* lse, cudaStream_t st) {
  const long blocks = (a.tc ? 0 : (long)a.nsp * a.Hkv * a.mtp) + (long)a.nso * a.B * a.Hkv * a.mto;
  if (blocks > 0x7fffffffl || (long)a.nsp * a.Hkv * a.mtp > 0x7fffffffl || (long)a.B * a.Hq > 0x7fffffffl)
    return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (a.direct) {
    CUDA_TRY(once_per_device((const void*)prefix_part_kernel<HD, QT, true>, [](int) {
      return cudaFuncSetAttribute(prefix_part_kernel<HD, QT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  pa_smem<HD>());
    }));
    CUDA_TRY(launch_k(prefix_part_kernel<HD, QT, true>, dim3((unsigned)(a.B * a.Hkv * a.mto)), PA_WARPS * 32,
                      (size_t)pa_smem<HD>(), st, a, o, ldo, lse));
    LAUNCH_CHECK();
    return GPT2_OK;
  }
  if (blocks) {
    CUDA_TRY(once_per_device((const void*)prefix_part_kernel<HD, QT, false>, [](int) {
      return cudaFuncSetAttribute(prefix_part_kernel<HD, QT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  pa_smem<HD>());
    }));
    CUDA_TRY(launch_k(prefix_part_kernel<HD, QT, false>, dim3((unsigned)blocks), PA_WARPS * 32, (size_t)pa_smem<HD>(), st,
                      a, o, ldo, lse));
    LAUNCH_CHECK();
  }
  if constexpr (HD >= 64 && sizeof(QT) == 2) {
    if (a.tc) {
      const int rc = (long)a.B * a.G <= 128 ? prefix_tc_run<HD, 1>(a, st) : prefix_tc_run<HD, 2>(a, st);
      if (rc != GPT2_OK) return rc;
    }
  }
  CUDA_TRY(launch_k(prefix_join_kernel<HD>, dim3((unsigned)(a.B * a.Hq)), 128, 0, st, a, o, ldo, lse));
  LAUNCH_CHECK();
  return GPT2_OK;
}

}  // namespace

size_t prefix_scratch_bytes(int B, int Hq, int Hkv, int hd, int P, int max_len) {
  PrefixPlan p;
  return prefix_plan(B, Hq, Hkv, hd, P, max_len, &p) ? p.bytes : 0;
}

int prefix_attention(const PrefixAttn& c, cudaStream_t st) {
  PrefixPlan p;
  if (!prefix_plan(c.B, c.Hq, c.Hkv, c.hd, c.P, c.max_len, &p)) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (c.q_f32 && p.tc) return GPT2_ERR_UNSUPPORTED_SHAPE;  // (a decode step has no 48 rows)
  if (c.scratch_bytes < p.bytes) return GPT2_ERR_WORKSPACE;
  PrefixArgs a = {};
  a.q = c.q; a.ldq = c.ldq; a.q_aligned = c.ldq % 8 == 0 && ((uintptr_t)c.q & 15) == 0;
  a.pk = reinterpret_cast<const bf16*>(c.pk); a.pv = reinterpret_cast<const bf16*>(c.pv);
  a.P = c.P; a.pcap = c.pcap;
  a.k = reinterpret_cast<const bf16*>(c.k); a.v = reinterpret_cast<const bf16*>(c.v);
  a.len = c.len; a.len_add = c.len_add; a.max_len = c.max_len;
  a.B = c.B; a.Hq = c.Hq; a.Hkv = c.Hkv; a.G = c.Hq / c.Hkv;
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)c.hd);
  a.direct = p.direct; a.tc = p.tc; a.Lp = p.Lp; a.Lo = p.Lo; a.nsp = p.nsp; a.nso = p.nso; a.mtp = p.mtp; a.mto = p.mto;
  a.po = reinterpret_cast<float*>(c.scratch);
  a.pml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(c.scratch) + p.po_bytes);
  bf16* o = reinterpret_cast<bf16*>(c.o);
  if (c.hd == 16)
    return c.q_f32 ? prefix_run<16, float>(a, o, c.ldo, c.lse, st) : prefix_run<16, bf16>(a, o, c.ldo, c.lse, st);
  if (c.hd == 64)
    return c.q_f32 ? prefix_run<64, float>(a, o, c.ldo, c.lse, st) : prefix_run<64, bf16>(a, o, c.ldo, c.lse, st);
  return c.q_f32 ? GPT2_ERR_UNSUPPORTED_SHAPE : prefix_run<128, bf16>(a, o, c.ldo, c.lse, st);
}

int prefix_attention_f32(const float* q, const float* pk, const float* pv, int P, long pcap, const float* k,
                         const float* v, const int32_t* len, int len_add, int max_len, int B, int H, int hd, float* o,
                         cudaStream_t st) {
  const dim3 grid(H, B);
  const float scale = 1.f / sqrtf((float)hd);
  if (hd == 64)
    CUDA_TRY(launch_k(prefix_f32_kernel<64>, grid, 32, 0, st, q, pk, pv, P, pcap, k, v, len, len_add, max_len, H, scale,
                      o));
  else if (hd == 16)
    CUDA_TRY(launch_k(prefix_f32_kernel<16>, grid, 32, 0, st, q, pk, pv, P, pcap, k, v, len, len_add, max_len, H, scale,
                      o));
  else
    return GPT2_ERR_UNSUPPORTED_SHAPE;
  LAUNCH_CHECK();
  return GPT2_OK;
}

int prefix_set_wait_limit(unsigned long long ns) {
  return set_unit_wait_limit(ns) == 0 ? GPT2_OK : GPT2_ERR_CUDA;
}

extern "C" {

size_t gpt2_op_prefix_attention_scratch_bytes(int B, int Hq, int Hkv, int hd, int prefix_len, int max_len) {
  return prefix_scratch_bytes(B, Hq, Hkv, hd, prefix_len, max_len);
}

int gpt2_op_prefix_attention_bf16(const uint16_t* q, int ldq, const uint16_t* pk, const uint16_t* pv, int prefix_len,
                                  int prefix_cap, const uint16_t* k, const uint16_t* v, const int32_t* len, int max_len,
                                  uint16_t* o, int ldo, float* lse, void* scratch, size_t scratch_bytes, int B, int Hq,
                                  int Hkv, int hd, void* stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || prefix_len < 0 || prefix_cap < prefix_len || max_len < 0)
    return GPT2_ERR_INVALID_ARG;
  if (B && (!q || !o || !scratch || (prefix_len && (!pk || !pv)) || (max_len && (!k || !v || !len))))
    return GPT2_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)o | (uintptr_t)lse | (uintptr_t)len) & 3) return GPT2_ERR_INVALID_ARG;
  if ((((uintptr_t)pk | (uintptr_t)pv) & 15 && prefix_len) || (((uintptr_t)k | (uintptr_t)v) & 15 && max_len))
    return GPT2_ERR_INVALID_ARG;
  if ((uintptr_t)scratch & 15) return GPT2_ERR_INVALID_ARG;
  if (hd != 16 && hd != 64 && hd != 128) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (Hq % Hkv) return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (ldq < (long)Hq * hd || ldo < (long)Hq * hd || ldq % 2 || ldo % 2) return GPT2_ERR_INVALID_ARG;
  if (B == 0) return GPT2_OK;
  PrefixAttn c = {};
  c.q = q; c.ldq = ldq; c.pk = pk; c.pv = pv; c.P = prefix_len; c.pcap = prefix_cap;
  c.k = k; c.v = v; c.len = len; c.max_len = max_len;
  c.o = o; c.ldo = ldo; c.lse = lse; c.scratch = scratch; c.scratch_bytes = scratch_bytes;
  c.B = B; c.Hq = Hq; c.Hkv = Hkv; c.hd = hd;
  return prefix_attention(c, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
