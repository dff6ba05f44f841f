// A serving step's tables built on the GPU from request lengths (sm_103a).
//
// Given each request's cached length and the number of tokens that the step adds to it,
// two launches leave everything that append and attention read: the pages of the new
// positions (taken from a reference-counted pool, lowest free ids first, as the host pool
// hands them out), the token lists and the per-token table rows, lengths and slots.
//
//   k_batch_admit  one cluster of 8 CTAs: finished requests give their pages back, the
//                  requests that fit are admitted, their pages are taken, the token lists
//                  are written.  The phases need each other's totals; a cluster has a
//                  hardware barrier and reads its neighbours' shared memory, so they take
//                  one launch and no wait on a flag in global memory.
//   k_batch_rows   the whole GPU: every token's table row, length and slot.  Bound by the
//                  T x max_pages row writes.  Launched as a programmatic dependent, so its
//                  launch overlaps the first kernel.
#include <climits>

#include "kernels.cuh"

namespace pa {

constexpr int kBatchCtas = 8;       // portable cluster size
constexpr int kBatchThreads = 1024;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// the 32-bit word at the address of `p` in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ int ld_cluster(const int *p, int rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Inclusive block scan of two 64-bit sums; *ta and *tb get the block totals.
__device__ void scan2(long long &a, long long &b, long long (*sh)[2], long long *ta,
                      long long *tb) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sh[w][0] = a;
    sh[w][1] = b;
  }
  __syncthreads();
  if (w == 0) {
    long long x = sh[lane][0], y = sh[lane][1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    sh[lane][0] = x;
    sh[lane][1] = y;
  }
  __syncthreads();
  if (w > 0) {
    a += sh[w - 1][0];
    b += sh[w - 1][1];
  }
  *ta = sh[31][0];
  *tb = sh[31][1];
  __syncthreads();
}

// First index in [0, n) whose value is greater than x (n if none); v is non-decreasing.
__device__ __forceinline__ int first_above(const int *v, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Pages that hold `len` positions.
__device__ __forceinline__ int pages_of(long long len, int P) { return (int)((len + P - 1) / P); }

__global__ void __launch_bounds__(kBatchThreads, 1)
k_batch_admit(BatchArgs a) {
  extern __shared__ int dyn[];
  int *pend = dyn;            // [n_seq] pages that requests 0..i need together (saturated)
  int *tend = dyn + a.n_seq;  // [n_seq] tokens that they add together (saturated)
  __shared__ long long sh[32][2];
  __shared__ int n_free_slice;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x;  // the grid is one cluster
  const long long cap = (long long)a.max_pages * a.P;

  // 1. page and token sums over the requests.  Every CTA does this for itself: the sums are
  //    then in its own shared memory, and n_seq is small beside a cluster barrier's cost.
  long long need_all = 0, toks_all = 0;
  int any_finished = 0;
  for (int i0 = 0; i0 < a.n_seq; i0 += kBatchThreads) {
    const int i = i0 + tid;
    long long need = 0, add = 0;
    if (i < a.n_seq) {
      const long long len = a.seq_len[i], nw = a.new_len[i];
      any_finished |= nw < 0;
      if (nw > 0) {
        if (len < 0 || len + nw > cap) {
          if (rank == 0 && a.err) atomicOr(a.err, PA_ERR_SEQ_RANGE);
        } else {
          need = pages_of(len + nw, a.P) - pages_of(len, a.P);
          add = nw;
        }
      }
    }
    long long tn, tt;
    scan2(need, add, sh, &tn, &tt);
    if (i < a.n_seq) {
      pend[i] = (int)min(need_all + need, (long long)INT_MAX);
      tend[i] = (int)min(toks_all + add, (long long)INT_MAX);
    }
    need_all += tn;
    toks_all += tt;
  }

  // 2. finished requests: a warp per row; each entry's page loses one reference
  if (__syncthreads_or(any_finished)) {
    for (int i = rank * (kBatchThreads / 32) + warp; i < a.n_seq;
         i += kBatchCtas * (kBatchThreads / 32)) {
      if (a.new_len[i] >= 0) continue;
      int32_t *row = a.seq_pt + (size_t)i * a.max_pages;
      for (int c = lane; c < a.max_pages; c += 32) {
        const int page = row[c];
        if (page < 0) continue;
        row[c] = -1;
        if (page >= a.num_pages) {
          if (a.err) atomicOr(a.err, PA_ERR_PAGE_RANGE);
        } else if (atomicSub(&a.page_ref[page], 1) <= 0) {
          // it was free already: no reference to give back (the order of two such
          // releases does not matter, each restores what it took)
          atomicAdd(&a.page_ref[page], 1);
          if (a.err) atomicOr(a.err, PA_ERR_REFCOUNT);
        }
      }
    }
    __threadfence();
    cluster_sync();  // the counts below see every release (they read past L1)
  }

  // 3. free pages.  CTA r owns a contiguous slice of the pool and a thread a contiguous
  //    piece of the slice, so one block scan ranks every free page by id.
  const int per_thread = (int)(((long long)a.num_pages + kBatchCtas * kBatchThreads * 4 - 1) /
                               (kBatchCtas * kBatchThreads * 4)) * 4;
  const long long g0 = ((long long)rank * kBatchThreads + tid) * per_thread;
  const int p0 = (int)min(g0, (long long)a.num_pages);
  const int p1 = (int)min(g0 + per_thread, (long long)a.num_pages);
  int rank0 = 0;       // free pages before this thread's
  long long free_all = 0;
  if (need_all > 0) {
    long long mine = 0, zero = 0, total, unused;
    int p = p0;
    for (; p + 4 <= p1; p += 4) {
      const int4 v = __ldcg(reinterpret_cast<const int4 *>(a.page_ref + p));
      mine += (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
    }
    for (; p < p1; ++p) mine += __ldcg(a.page_ref + p) == 0;
    long long incl = mine;
    scan2(incl, zero, sh, &total, &unused);
    if (tid == 0) n_free_slice = (int)total;
    cluster_sync();
    long long before = 0;
    for (int r = 0; r < kBatchCtas; ++r) {
      const int n = ld_cluster(&n_free_slice, r);
      if (r < rank) before += n;
      free_all += n;
    }
    rank0 = (int)(before + incl - mine);
  }

  // 4. the longest prefix of the requests whose pages and tokens fit
  const int n_fit_pages = first_above(pend, a.n_seq, (int)min(free_all, (long long)INT_MAX - 1));
  const int n_fit_toks = first_above(tend, a.n_seq, min(a.T, INT_MAX - 1));
  const int n_adm = min(n_fit_pages, n_fit_toks);
  const int n_take = n_adm > 0 ? pend[n_adm - 1] : 0;
  const int n_tok = n_adm > 0 ? tend[n_adm - 1] : 0;
  if (rank == 0 && tid == 0 && a.err && (n_tok < toks_all)) atomicOr(a.err, PA_ERR_NO_SPACE);

  // 5. the r-th free page goes to the request whose page range holds r
  if (n_take > rank0) {
    int r = rank0, i = -1, i_end = 0, i_beg = 0, first = 0;
    for (int p = p0; p < p1 && r < n_take; ++p) {
      if (__ldcg(a.page_ref + p) != 0) continue;
      if (i < 0 || r >= i_end) {
        i = first_above(pend, n_adm, r);
        i_end = pend[i];
        i_beg = i > 0 ? pend[i - 1] : 0;
        first = pages_of(a.seq_len[i], a.P);
      }
      a.seq_pt[(size_t)i * a.max_pages + first + (r - i_beg)] = p;
      a.page_ref[p] = 1;
      ++r;
    }
  }

  // 6. first token of every request, then the tokens' requests and positions
  const int g = rank * kBatchThreads + tid, stride = kBatchCtas * kBatchThreads;
  for (int i = g; i <= a.n_seq; i += stride)
    a.q_start[i] = i == 0 || n_adm == 0 ? 0 : tend[min(i, n_adm) - 1];
  for (int t = g; t < a.T; t += stride) {
    int s = -1, pos = 0;
    if (t < n_tok) {
      s = first_above(tend, n_adm, t);
      pos = a.seq_len[s] + t - (s > 0 ? tend[s - 1] : 0);
    }
    a.tok_seq[t] = s;
    a.tok_pos[t] = pos;
    a.tok_kv[t] = s < 0 ? 0 : pos + 1;
  }
  // a CTA's shared memory stays until its neighbours have read its free-page count
  if (need_all > 0) cluster_sync();
}

// Every token's table row and slot.  A warp takes kTok consecutive tokens: tokens of one
// request (a prompt's chunk) share a row, which is then read once and written kTok times.
template <typename V, int kTok>
__global__ void __launch_bounds__(256)
k_batch_rows(BatchArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int nwarps = (gridDim.x * blockDim.x) >> 5;
  constexpr int kPer = sizeof(V) / 4;
  const int n_vec = a.max_pages / kPer;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.n_seq; i += gridDim.x * blockDim.x)
    a.seq_len_out[i] = a.new_len[i] < 0 ? 0 : a.seq_len[i] + (a.q_start[i + 1] - a.q_start[i]);
  V pad;
#pragma unroll
  for (int e = 0; e < kPer; ++e) reinterpret_cast<int *>(&pad)[e] = -1;
  for (long long t0 = (long long)warp * kTok; t0 < a.T; t0 += (long long)nwarps * kTok) {
    int seq[kTok];
    bool same = true;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      seq[j] = t0 + j < a.T ? a.tok_seq[t0 + j] : -2;
      same = same && seq[j] == seq[0];
    }
    if (lane < kTok && t0 + lane < a.T) {
      const int s = a.tok_seq[t0 + lane], pos = a.tok_pos[t0 + lane];
      const int page = s < 0 ? -1 : a.seq_pt[(size_t)s * a.max_pages + pos / a.P];
      a.slot[t0 + lane] = page < 0 ? -1 : (int64_t)page * a.P + pos % a.P;
    }
    for (int j = 0; j < kTok; ++j) {
      if (seq[j] == -2) break;
      const V *src = reinterpret_cast<const V *>(a.seq_pt + (size_t)max(seq[j], 0) * a.max_pages);
      V *dst = reinterpret_cast<V *>(a.tok_pt + (size_t)(t0 + j) * a.max_pages);
      const int copies = same ? kTok : 1;
#pragma unroll 4
      for (int c = lane; c < n_vec; c += 32) {
        const V v = seq[j] < 0 ? pad : src[c];
        for (int k = 0; k < copies; ++k) dst[(size_t)k * n_vec + c] = v;
      }
      if (same) break;
    }
  }
}

template <typename V>
static cudaError_t launch_rows(const BatchArgs &a, int num_sms, cudaStream_t s) {
  // four tokens a warp once every SM has its eight CTAs' warps full of them
  const bool many = a.T >= num_sms * 64 * 4;
  const long long warps = many ? (a.T + 3) / 4 : a.T;
  long long blocks = (warps + 7) / 8, need_seq = (a.n_seq + 255) / 256;
  if (blocks < need_seq) blocks = need_seq;
  if (blocks > (long long)num_sms * 8) blocks = (long long)num_sms * 8;
  if (blocks < 1) blocks = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, k_batch_rows<V, 4>, a)
              : cudaLaunchKernelEx(&cfg, k_batch_rows<V, 1>, a);
}

cudaError_t launch_batch(const BatchArgs &a, int num_sms, cudaStream_t s) {
  const size_t smem = (size_t)a.n_seq * 8;
  static PerDeviceOnce setup;
  if (setup.first()) {
    cudaError_t e = cudaFuncSetAttribute(k_batch_admit, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBatchMaxSeq * 8);
    if (e != cudaSuccess) return e;
    setup.mark();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kBatchCtas);
  cfg.blockDim = dim3(kBatchThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBatchCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_batch_admit, a);
  if (e != cudaSuccess) return e;
  return a.max_pages % 4 == 0 ? launch_rows<int4>(a, num_sms, s) : launch_rows<int>(a, num_sms, s);
}

}  // namespace pa
