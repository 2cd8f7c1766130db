// Rules on the logits of a decode step, with the greedy choice of what they
// leave: penalties for tokens that occurred before, biases, a grammar's mask.
//
//   z1 = v seen in the history ? (z > 0 ? z / rep : z rep) : z
//   z2 = (z1 - freq c) - (c > 0 ? pres : 0),  c = occurrences of v among the generated tokens
//   z3 = z2 + bias[v]
//   z4 = allowed[v] ? z3 : -inf
//   next = argmax z4 (lowest id among equal maxima)
//
// every step rounded to fp32 on its own (no fused multiply-add), so that the
// choice does not depend on how the kernel is arranged.
#include "common.cuh"
#include "internal.h"

namespace {

constexpr int RL_THREADS = 512;
constexpr int RL_MAX_SPLIT = 8;          // blocks of a row (a cluster)
constexpr int RL_MAX_SLICE = 49152;      // ids of a block: one counter word each in shared memory
constexpr int RL_MAX_BIAS = 4096;
constexpr uint32_t RL_SEEN = 0x80000000u;  // in the history, not among the generated tokens
constexpr uint32_t RL_BIAS = 0x40000000u;  // has a bias entry; the low 30 bits count

struct RulesArgs {
  const float* z;
  long ld;
  float* out;
  long ldo;
  int V, per, split;  // ids of a block (a multiple of 32), blocks of a row
  gpt2_logit_rules r;
  int counted, n_bias;
  int32_t* next;
  int32_t* pos;
};

struct RowRules {
  float rep, pres, freq;
};
DEVI float penalised(float z, uint32_t w, const RowRules& p) {
  if (w & ~RL_BIAS) {
    z = z > 0.f ? __fdiv_rn(z, p.rep) : __fmul_rn(z, p.rep);
    const uint32_t c = w & (RL_BIAS - 1);
    if (c) {
      z = __fsub_rn(z, __fmul_rn(p.freq, (float)c));
      z = __fsub_rn(z, p.pres);
    }
  }
  return z;
}

// One row's slice of ids.  Bound by the logits' way in and out of HBM at large
// batches, by latency at small ones, where a cluster of blocks shares the
// row.  Each block counts the history's tokens of its own slice in shared
// memory (integer additions: the order of the atomics does not matter), so
// no counters are kept, zeroed or joined in global memory; the first batch
// of logits is requested before that.  Ids with a bias entry are left out of
// the pass and finished by the thread of their last entry.
__global__ void __launch_bounds__(RL_THREADS) logit_rules_kernel(const __grid_constant__ RulesArgs a) {
  extern __shared__ uint32_t rl_cnt[];  // [per] counters, then [n_bias] bias ids
  __shared__ float sv[RL_THREADS / 32];
  __shared__ int si[RL_THREADS / 32];
  constexpr int U = 8;  // loads in flight per thread
  const int rank = a.split > 1 ? (int)cluster_ctarank() : 0;
  const int row = blockIdx.x / a.split, tid = threadIdx.x;
  const int v0 = rank * a.per, nv = max(0, min(a.per, a.V - v0));
  const float* z = a.z + (size_t)row * a.ld + v0;
  float* out = a.out + (size_t)row * a.ldo + v0;
  pdl_trigger();
  if (a.counted)
    for (int i = tid; i < nv; i += RL_THREADS) rl_cnt[i] = 0;
  pdl_wait();
  float x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = tid + u * RL_THREADS;
    x[u] = i < nv ? z[i] : -INFINITY;
  }
  RowRules p = {1.f, 0.f, 0.f};
  if (a.r.repetition) p.rep = a.r.repetition[row];
  if (a.r.presence) p.pres = a.r.presence[row];
  if (a.r.frequency) p.freq = a.r.frequency[row];
  int hn = 0;
  int* bid = reinterpret_cast<int*>(rl_cnt + a.per);
  if (a.counted) {
    if (a.r.history) {
      hn = a.r.history_len[row];
      hn = hn < 0 ? 0 : (hn > a.r.history_ld ? a.r.history_ld : hn);
    }
    const int g0 = a.r.gen_start ? a.r.gen_start[row] : 0;
    const int32_t* hist = a.r.history + (size_t)row * a.r.history_ld;
    const int32_t* ids = a.r.bias_ids + (size_t)row * a.n_bias;
    __syncthreads();
    for (int i0 = tid; i0 < hn; i0 += U * RL_THREADS) {
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * RL_THREADS;
        id[u] = i < hn ? hist[i] - v0 : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * RL_THREADS;
        if (id[u] >= 0 && id[u] < nv) {  // ids outside the vocabulary are nobody's
          if (i >= g0) atomicAdd(&rl_cnt[id[u]], 1u);
          else atomicOr(&rl_cnt[id[u]], RL_SEEN);
        }
      }
    }
    for (int e = tid; e < a.n_bias; e += RL_THREADS) {
      const int id = ids[e] - v0;
      bid[e] = id;
      if (id >= 0 && id < nv) atomicOr(&rl_cnt[id], RL_BIAS);
    }
    __syncthreads();
  }
  const uint32_t* allowed = a.r.allowed ? a.r.allowed + (size_t)row * a.r.allowed_ld + (v0 >> 5) : nullptr;
  float bv = -INFINITY;
  int bi = 0x7fffffff;
  for (int i0 = tid; i0 < nv; i0 += U * RL_THREADS) {
    float y[U];
    uint32_t w[U], m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RL_THREADS;
      y[u] = x[u];
      w[u] = a.counted && i < nv ? rl_cnt[i] : 0u;
      m[u] = allowed && i < nv ? allowed[i >> 5] : 0xffffffffu;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {  // the next batch
      const int i = i0 + (U + u) * RL_THREADS;
      x[u] = i < nv ? z[i] : -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RL_THREADS;
      if (i >= nv || (w[u] & RL_BIAS)) continue;
      const float t = (m[u] >> (i & 31)) & 1u ? penalised(y[u], w[u], p) : -INFINITY;
      out[i] = t;
      if (t > bv || (t != t && bv == bv)) {  // a thread meets its ids in rising order
        bv = t;
        bi = v0 + i;
      }
    }
  }
  for (int e = tid; e < a.n_bias; e += RL_THREADS) {
    const int i = bid[e];
    if (i < 0 || i >= nv) continue;
    bool last = true;  // of several entries of an id the last one counts
    for (int f = e + 1; f < a.n_bias; ++f) last = last && bid[f] != i;
    if (!last) continue;
    float t = -INFINITY;
    if (!allowed || (allowed[i >> 5] >> (i & 31)) & 1u)
      t = __fadd_rn(penalised(z[i], rl_cnt[i], p), a.r.bias_values[(size_t)row * a.n_bias + e]);
    out[i] = t;
    if (greedy_better(t, v0 + i, bv, bi)) {
      bv = t;
      bi = v0 + i;
    }
  }
  if (!a.next) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
    const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
    if (greedy_better(ov, oi, bv, bi)) {
      bv = ov;
      bi = oi;
    }
  }
  if ((tid & 31) == 0) {
    sv[tid >> 5] = bv;
    si[tid >> 5] = bi;
  }
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < RL_THREADS / 32; ++k)
      if (greedy_better(sv[k], si[k], bv, bi)) {
        bv = sv[k];
        bi = si[k];
      }
    sv[0] = bv;
    si[0] = bi;
  }
  if (a.split > 1) cluster_sync_all();
  if (rank == 0 && tid == 0) {
    for (int k = 1; k < a.split; ++k) {
      float ov;
      int oi;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(ov) : "r"(mapa_shared(smem_u32(sv), k)) : "memory");
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(oi) : "r"(mapa_shared(smem_u32(si), k)) : "memory");
      if (greedy_better(ov, oi, bv, bi)) {
        bv = ov;
        bi = oi;
      }
    }
    const int32_t id = bi < a.V ? bi : 0;  // nothing above -inf: id 0, as gpt2_greedy_next
    a.next[row] = id;
    if (a.pos) a.pos[row] += 1;
    // (every block of the row has read the history: they met above)
    if (a.r.append && hn < a.r.history_ld) {
      a.r.history[(size_t)row * a.r.history_ld + hn] = id;
      a.r.history_len[row] = hn + 1;
    }
  }
  if (a.split > 1) cluster_sync_all();  // no block leaves while rank 0 reads it
}

bool bad_align(const void* p) { return ((uintptr_t)p & 3) != 0; }

}  // namespace

int logit_rules(const float* logits, long ld, float* out, long ldo, int rows, int vocab, const gpt2_logit_rules* r,
                int32_t* next, int32_t* pos, cudaStream_t st) {
  if (!logits || !out || !r || rows < 0 || vocab < 0 || ld < vocab || ldo < vocab) return GPT2_ERR_INVALID_ARG;
  if (logits == out && ld != ldo) return GPT2_ERR_INVALID_ARG;
  if (pos && !next) return GPT2_ERR_INVALID_ARG;
  if (r->history && (!r->history_len || r->history_ld < 1)) return GPT2_ERR_INVALID_ARG;
  if (r->append && (!r->history || !next)) return GPT2_ERR_INVALID_ARG;
  if (r->n_bias < 0 || (r->n_bias && (!r->bias_ids || !r->bias_values))) return GPT2_ERR_INVALID_ARG;
  if (r->allowed && r->allowed_ld < (vocab + 31) / 32) return GPT2_ERR_INVALID_ARG;
  if (bad_align(logits) || bad_align(out) || bad_align(r->history) || bad_align(r->history_len) ||
      bad_align(r->gen_start) || bad_align(r->repetition) || bad_align(r->presence) || bad_align(r->frequency) ||
      bad_align(r->bias_ids) || bad_align(r->bias_values) || bad_align(r->allowed) || bad_align(next) || bad_align(pos))
    return GPT2_ERR_INVALID_ARG;
  if (vocab > RL_MAX_SPLIT * RL_MAX_SLICE - 32 * RL_MAX_SPLIT || r->n_bias > RL_MAX_BIAS || rows > (1 << 27))
    return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || vocab == 0) return GPT2_OK;
  RulesArgs a = {};
  a.z = logits; a.ld = ld; a.out = out; a.ldo = ldo; a.V = vocab; a.r = *r; a.next = next; a.pos = pos;
  a.n_bias = r->n_bias;
  a.counted = r->history || r->n_bias;
  // blocks of a row: 8 while that fits the machine at once, and enough that
  // the counters of four blocks fit an SM
  int split = 1;
  while (split < RL_MAX_SPLIT && ((long)rows * split * 2 <= 4l * num_sms() || (vocab + split - 1) / split > 12800))
    split *= 2;
  a.split = split;
  a.per = ((vocab + split - 1) / split + 31) / 32 * 32;
  const size_t smem = a.counted ? (size_t)a.per * 4 + (size_t)a.n_bias * 4 : 0;
  CUDA_TRY(once_per_device((const void*)logit_rules_kernel, [](int) {
    return cudaFuncSetAttribute(logit_rules_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (RL_MAX_SLICE + RL_MAX_BIAS) * 4);
  }));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * split));
  cfg.blockDim = dim3(RL_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, logit_rules_kernel, a));
  LAUNCH_CHECK();
  return GPT2_OK;
}

extern "C" {

int gpt2_op_logit_rules(const float* logits, int ld, float* out, int ldo, int rows, int vocab,
                        const gpt2_logit_rules* rules, int32_t* next, int32_t* pos, void* stream) {
  return logit_rules(logits, ld, out, ldo, rows, vocab, rules, next, pos, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
