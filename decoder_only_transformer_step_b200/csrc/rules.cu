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

constexpr int RL_THREADS = 256;
constexpr int RL_MAX_SPLIT = 8;          // blocks of a row (a cluster)
constexpr int RL_MAX_SLICE = 32768;      // ids of a block: a word each in shared memory, and their list
constexpr int RL_MAX_BIAS = 4095;
constexpr int RL_MAX_HISTORY = (1 << 18) - 1;
// An id's word: bit 31 where it is in the history before gen_start, bits
// 18..29 the place of its last bias entry (1 ..), bits 0..17 its occurrences
// among the generated ids.  0: no rule but the mask touches it.
constexpr uint32_t RL_SEEN = 0x80000000u, RL_COUNT = (1u << 18) - 1;

struct RulesArgs {
  const float* z;
  long ld;
  float* out;
  long ldo;
  int V, per, split;  // ids of a block (a multiple of 32), blocks of a row
  gpt2_logit_rules r;
  int n_bias, list;   // list: room for the ids with a word (COUNTED)
  int32_t* next;
  int32_t* pos;
  int* err;  // device status word or NULL
};

// One row's slice of ids.  Bound by the logits' way in and out of HBM at large
// batches, by latency at small ones, where a cluster of blocks shares the
// row.  Each block notes its own slice's bias entries and history in shared
// memory (integer maxima, sums and ors: the order of the atomics does not
// matter), so nothing is kept, zeroed or joined in global memory; the first
// batch of logits is requested before that.  The pass over the slice only
// masks, copies and compares; the few ids with a word are listed and left to a
// second pass with a thread each, since in the first almost every warp would
// take their path for one lane.  384 x 50257 with histories of 4096 ids: 63 us
// (logits in and out at 2.5 TB/s, issue slots 65 % busy), 42 without a history,
// 36 without biases too, 27 without mask and choice as well; 16 x 50257: 7.2 us, one
// round trip after the other: lengths and history, mask, listed ids, exchange.
template <bool COUNTED, bool MASKED>
__global__ void __launch_bounds__(RL_THREADS) logit_rules_kernel(const __grid_constant__ RulesArgs a) {
  extern __shared__ __align__(16) uint32_t rl_word[];  // [per] words, [n_bias] bias values, [list] ids
  __shared__ float sv[RL_THREADS / 32];
  __shared__ int si[RL_THREADS / 32];
  __shared__ int listed;
  __shared__ __align__(8) uint64_t best[RL_MAX_SPLIT], arrived;
  constexpr int U = 8, UH = 8;  // loads of logits / of history in flight per thread
  const int rank = a.split > 1 ? (int)cluster_ctarank() : 0;
  const int row = blockIdx.x / a.split, tid = threadIdx.x;
  const int v0 = rank * a.per, nv = max(0, min(a.per, a.V - v0));
  const float* z = a.z + (size_t)row * a.ld + v0;
  float* out = a.out + (size_t)row * a.ldo + v0;
  float* bias = reinterpret_cast<float*>(rl_word + a.per);
  uint16_t* list = reinterpret_cast<uint16_t*>(bias + a.n_bias);
  pdl_trigger();
  // the row's blocks report to rank 0 (below): its barrier is set up first
  const bool meets = a.next && a.split > 1;
  if (meets) {
    if (rank == 0 && tid == 0) {
      mbar_init(smem_u32(&arrived), 1);
      mbar_fence_init();
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  if constexpr (COUNTED) {
    if (tid == 0) listed = 0;
    for (int i = tid; i < a.per / 4; i += RL_THREADS) reinterpret_cast<uint4*>(rl_word)[i] = make_uint4(0, 0, 0, 0);
  }
  pdl_wait();
  // requested here, ahead of the phases below: the row's lengths, its first
  // history and bias entries, its first logits (the mask's words and the
  // penalties are requested where they are used, the listed ids' logits again)
  int hn = 0, g0 = 0, be = -1, h0[UH];
  float bval = 0.f;
  const size_t brow = (size_t)row * a.n_bias;
  const int32_t* hist = a.r.history + (size_t)row * a.r.history_ld;
  if constexpr (COUNTED) {
    if (a.r.history) hn = a.r.history_len[row];
    if (a.r.gen_start) g0 = a.r.gen_start[row];
#pragma unroll
    for (int u = 0; u < UH; ++u) {
      const int i = tid + u * RL_THREADS;
      h0[u] = a.r.history && i < a.r.history_ld ? hist[i] : -1;
    }
    if (tid < a.n_bias) {
      be = a.r.bias_ids[brow + tid];
      bval = a.r.bias_values[brow + tid];
    }
  }
  float x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = tid + u * RL_THREADS;
    x[u] = i < nv ? z[i] : -INFINITY;
  }
  if constexpr (COUNTED) {
    hn = a.r.history ? (hn < 0 ? 0 : (hn > a.r.history_ld ? a.r.history_ld : hn)) : 0;
    __syncthreads();
    if (a.n_bias) {
      for (int e = tid; e < a.n_bias; e += RL_THREADS) {
        if (e != tid) {
          be = a.r.bias_ids[brow + e];
          bval = a.r.bias_values[brow + e];
        }
        const int id = be - v0;
        bias[e] = bval;
        // the last entry stays
        if (id >= 0 && id < nv && atomicMax(&rl_word[id], (uint32_t)(e + 1) << 18) == 0)
          list[atomicAdd(&listed, 1)] = (uint16_t)id;
      }
      __syncthreads();
    }
    for (int i0 = tid; i0 < hn; i0 += UH * RL_THREADS) {
      if (i0 != tid) {
#pragma unroll
        for (int u = 0; u < UH; ++u) {
          const int i = i0 + u * RL_THREADS;
          h0[u] = i < hn ? hist[i] : -1;
        }
      }
#pragma unroll
      for (int u = 0; u < UH; ++u) {
        const int i = i0 + u * RL_THREADS, id = h0[u] - v0;
        if (i < hn && id >= 0 && id < nv) {  // (ids outside the vocabulary are nobody's)
          const uint32_t old = i >= g0 ? atomicAdd(&rl_word[id], 1u) : atomicOr(&rl_word[id], RL_SEEN);
          if (old == 0) list[atomicAdd(&listed, 1)] = (uint16_t)id;
        }
      }
    }
    __syncthreads();
  }
  const uint32_t* allowed = MASKED ? a.r.allowed + (size_t)row * a.r.allowed_ld + (v0 >> 5) : nullptr;
  const uint32_t bit = 1u << (tid & 31);  // (the stride of a thread's ids is a multiple of 32)
  float bv = -INFINITY;
  int bi = 0x7fffffff;
  auto finish = [&](int i, float t, uint32_t w, uint32_t m) {
    if (MASKED && !(m & bit)) t = -INFINITY;
    if (COUNTED && w) return;
    out[i] = t;
    if (!(t <= bv) && bv == bv) {  // larger, or the first NaN: a thread meets its ids in rising order
      bv = t;
      bi = i;
    }
  };
  int i0 = tid;
  for (; i0 + (U - 1) * RL_THREADS < nv; i0 += U * RL_THREADS) {
    float y[U];
    uint32_t w[U], m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      y[u] = x[u];
      w[u] = COUNTED ? rl_word[i0 + u * RL_THREADS] : 0u;
      m[u] = MASKED ? allowed[(i0 >> 5) + u * (RL_THREADS / 32)] : 0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {  // the next batch
      const int i = i0 + (U + u) * RL_THREADS;
      if (i < nv) x[u] = z[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) finish(i0 + u * RL_THREADS, y[u], w[u], m[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + u * RL_THREADS;
    if (i < nv) finish(i, x[u], COUNTED ? rl_word[i] : 0u, MASKED ? allowed[i >> 5] : 0u);
  }
  if (bi != 0x7fffffff) bi += v0;
  if constexpr (COUNTED) {
    const int n = listed;
    if (tid < n) {
      const float rep = a.r.repetition ? a.r.repetition[row] : 1.f, pres = a.r.presence ? a.r.presence[row] : 0.f,
                  freq = a.r.frequency ? a.r.frequency[row] : 0.f;
      for (int j = tid; j < n; j += RL_THREADS) {
        const int i = list[j];
        const uint32_t w = rl_word[i], c = w & RL_COUNT, e = (w >> 18) & 0xfffu;
        float t = z[i];
        if (c || (w & RL_SEEN)) t = t > 0.f ? __fdiv_rn(t, rep) : __fmul_rn(t, rep);
        if (c) t = __fsub_rn(__fsub_rn(t, __fmul_rn(freq, (float)c)), pres);
        if (e) t = __fadd_rn(t, bias[e - 1]);
        if (MASKED && !((allowed[i >> 5] >> (i & 31)) & 1u)) t = -INFINITY;
        out[i] = t;
        if (t != -INFINITY && greedy_better(t, v0 + i, bv, bi)) {  // (-inf is never chosen, as above)
          bv = t;
          bi = v0 + i;
        }
      }
    }
  }
  if (!a.next) return;
  __syncwarp();
  if (meets) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
    // Ranks above 0 send (value, id) into rank 0's shared memory, counted on
    // its barrier: no fence waits for this block's stores to HBM, and the
    // block may leave.  A row whose blocks do not meet in time has no choice:
    // id -1, which no later step takes for a token, and nothing moves on.
    if (rank > 0) {
      const uint64_t v = (uint64_t)(uint32_t)bi << 32 | __float_as_uint(bv);
      asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                       mapa_shared(smem_u32(&best[rank]), 0)),
                   "l"(v), "r"(mapa_shared(smem_u32(&arrived), 0))
                   : "memory");
    } else {
      if (a.split > 1) {
        const uint32_t bar = smem_u32(&arrived);
        mbar_arrive_expect_tx(bar, 8u * (a.split - 1));
        int gave_up = 0;
        if (!mbar_wait_bounded(bar, 0, &gave_up, a.err)) {
          mbar_drain_bounded(bar, 0);  // (the others still send into this block's memory)
          a.next[row] = -1;
          return;
        }
        for (int k = 1; k < a.split; ++k) {
          const uint64_t v = *reinterpret_cast<volatile uint64_t*>(&best[k]);
          const float ov = __uint_as_float((uint32_t)v);
          const int oi = (int)(v >> 32);
          if (greedy_better(ov, oi, bv, bi)) {
            bv = ov;
            bi = oi;
          }
        }
      }
      const int32_t id = bi < a.V ? bi : 0;  // nothing above -inf: id 0, as gpt2_greedy_next
      a.next[row] = id;
      if (a.pos) a.pos[row] += 1;
      // (every block of the row has read the history before it reported)
      if (a.r.append && hn < a.r.history_ld) {
        a.r.history[(size_t)row * a.r.history_ld + hn] = id;
        a.r.history_len[row] = hn + 1;
      }
    }
  }
}

template <bool COUNTED, bool MASKED>
int rules_launch(const RulesArgs& a, int rows, cudaStream_t st) {
  CUDA_TRY(once_per_device((const void*)logit_rules_kernel<COUNTED, MASKED>, [](int) {
    return cudaFuncSetAttribute(logit_rules_kernel<COUNTED, MASKED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                227 * 1024 - 256);
  }));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * a.split));
  cfg.blockDim = dim3(RL_THREADS);
  cfg.dynamicSmemBytes = COUNTED ? (size_t)a.per * 4 + (size_t)a.n_bias * 4 + (size_t)a.list * 2 : 0;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, logit_rules_kernel<COUNTED, MASKED>, a));
  LAUNCH_CHECK();
  return GPT2_OK;
}

bool bad_align(const void* p) { return ((uintptr_t)p & 3) != 0; }

}  // namespace

int rules_set_wait_limit(unsigned long long ns) { return set_unit_wait_limit(ns) == 0 ? GPT2_OK : GPT2_ERR_CUDA; }

int logit_rules(const float* logits, long ld, float* out, long ldo, int rows, int vocab, const gpt2_logit_rules* r,
                int32_t* next, int32_t* pos, int* err, cudaStream_t st) {
  if (!r || rows < 0 || vocab < 0 || ld < vocab || ldo < vocab) return GPT2_ERR_INVALID_ARG;
  const bool any = rows && vocab;  // (an empty tensor's address is NULL)
  if (any && (!logits || !out || (logits == out && ld != ldo))) return GPT2_ERR_INVALID_ARG;
  if (pos && !next) return GPT2_ERR_INVALID_ARG;
  if (r->history && (!r->history_len || r->history_ld < 1)) return GPT2_ERR_INVALID_ARG;
  if (r->append && any && (!r->history || !next)) return GPT2_ERR_INVALID_ARG;
  if (r->n_bias < 0 || (r->n_bias && any && (!r->bias_ids || !r->bias_values))) return GPT2_ERR_INVALID_ARG;
  if (r->allowed && r->allowed_ld < (vocab + 31) / 32) return GPT2_ERR_INVALID_ARG;
  if (bad_align(logits) || bad_align(out) || bad_align(r->history) || bad_align(r->history_len) ||
      bad_align(r->gen_start) || bad_align(r->repetition) || bad_align(r->presence) || bad_align(r->frequency) ||
      bad_align(r->bias_ids) || bad_align(r->bias_values) || bad_align(r->allowed) || bad_align(next) || bad_align(pos))
    return GPT2_ERR_INVALID_ARG;
  if (vocab > RL_MAX_SPLIT * RL_MAX_SLICE || r->n_bias > RL_MAX_BIAS ||
      (r->history && r->history_ld > RL_MAX_HISTORY) || rows > (1 << 27))
    return GPT2_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || vocab == 0) return GPT2_OK;
  RulesArgs a = {};
  a.z = logits; a.ld = ld; a.out = out; a.ldo = ldo; a.V = vocab; a.r = *r; a.next = next; a.pos = pos; a.err = err;
  a.n_bias = r->n_bias;
  // blocks of a row: 8 while that fits the machine at once, and enough that
  // the words of six blocks fit an SM
  int split = 1;
  while (split < RL_MAX_SPLIT && ((long)rows * split * 2 <= 6l * num_sms() || (vocab + split - 1) / split > 8192))
    split *= 2;
  a.split = split;
  a.per = ((vocab + split - 1) / split + 31) / 32 * 32;
  const long most = (r->history ? (long)r->history_ld : 0) + r->n_bias;  // ids that can have a word
  a.list = (int)(most < a.per ? most : a.per);
  if (most) return a.r.allowed ? rules_launch<true, true>(a, rows, st) : rules_launch<true, false>(a, rows, st);
  return a.r.allowed ? rules_launch<false, true>(a, rows, st) : rules_launch<false, false>(a, rows, st);
}

extern "C" {

int gpt2_op_logit_rules(const float* logits, int ld, float* out, int ldo, int rows, int vocab,
                        const gpt2_logit_rules* rules, int32_t* next, int32_t* pos, void* stream) {
  return logit_rules(logits, ld, out, ldo, rows, vocab, rules, next, pos, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
