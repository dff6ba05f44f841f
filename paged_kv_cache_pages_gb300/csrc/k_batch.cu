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
constexpr int kRounds = 64;         // at most: the pool's pieces of one warp

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

__device__ __forceinline__ int warp_incl(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Reference counts of pages p .. p + 3 of a pool of n; past its end: in use.
__device__ __forceinline__ int4 ref4(const int32_t *ref, int p, int n) {
  if (p + 4 <= n) return __ldcg(reinterpret_cast<const int4 *>(ref + p));
  return make_int4(p < n ? __ldcg(ref + p) : 1, p + 1 < n ? __ldcg(ref + p + 1) : 1,
                   p + 2 < n ? __ldcg(ref + p + 2) : 1, 1);
}

__global__ void __launch_bounds__(kBatchThreads, 1)
k_batch_admit(BatchArgs a) {
  extern __shared__ int dyn[];
  int *pend = dyn;               // [n_seq] pages that requests 0..i need together (saturated)
  int *tend = pend + a.n_seq;    // [n_seq] tokens that they add together (saturated)
  int *first = tend + a.n_seq;   // [n_seq] pages that request i has
  int *fin = first + a.n_seq;    // [n_fin] finished requests
  __shared__ long long sh[32][2];
  __shared__ int free_cnt[kRounds][32], free_cta[kRounds], free_base[kRounds];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x;  // the grid is one cluster
  constexpr int kWarps = kBatchCtas * kBatchThreads / 32;
  const int gw = rank * (kBatchThreads / 32) + warp;
  const long long cap = (long long)a.max_pages * a.P;

  // 1. page and token sums over the requests, and the list of the finished ones (counted in
  //    the token sum's upper bits: at most 2^13 requests of at most 2^30 tokens).  Every CTA
  //    does this for itself: the sums are then in its own shared memory, and n_seq is small
  //    beside a cluster barrier's cost.
  constexpr int kFinBit = 48;
  constexpr long long kTokMask = (1ll << kFinBit) - 1;
  long long need_all = 0, toks_all = 0;
  for (int i0 = 0; i0 < a.n_seq; i0 += kBatchThreads) {
    const int i = i0 + tid;
    long long need = 0, add = 0;
    bool end = false;
    if (i < a.n_seq) {
      const long long len = a.seq_len[i], nw = a.new_len[i];
      end = nw < 0;
      if (nw > 0) {
        if (len < 0 || len + nw > cap) {
          if (rank == 0 && a.err) atomicOr(a.err, PA_ERR_SEQ_RANGE);
        } else {
          first[i] = pages_of(len, a.P);
          need = pages_of(len + nw, a.P) - first[i];
          add = nw;
        }
      }
      if (end) add = 1ll << kFinBit;
    }
    long long tn, tt;
    scan2(need, add, sh, &tn, &tt);
    if (i < a.n_seq) {
      pend[i] = (int)min(need_all + need, (long long)INT_MAX);
      tend[i] = (int)min((toks_all + add) & kTokMask, (long long)INT_MAX);
      if (end) fin[(int)((toks_all + add) >> kFinBit) - 1] = i;
    }
    need_all += tn;
    toks_all += tt;
  }
  const int n_fin = (int)(toks_all >> kFinBit);
  toks_all &= kTokMask;
  __syncthreads();

  // 2. finished requests: each entry's page loses one reference.  The cluster's warps share
  //    the rows in pieces of 128 entries, four a lane, whose loads are in flight together,
  //    and the decrements return nothing; a page that had no reference left shows below zero
  //    in the next step.
  if (n_fin > 0) {
    const int pieces = (a.max_pages + 127) / 128;
    for (long long u = gw; u < (long long)n_fin * pieces; u += kWarps) {
      const int f = (int)(u / pieces), x = (int)(u - (long long)f * pieces);
      int32_t *row = a.seq_pt + (size_t)fin[f] * a.max_pages;
      int page[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = x * 128 + k * 32 + lane;
        page[k] = c < a.max_pages ? row[c] : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (page[k] < 0) continue;
        row[x * 128 + k * 32 + lane] = -1;
        if (page[k] < a.num_pages) atomicSub(&a.page_ref[page[k]], 1);
        else if (a.err) atomicOr(a.err, PA_ERR_PAGE_RANGE);
      }
    }
    __threadfence();
    cluster_sync();  // the counts below see every release (they read past L1)
  }

  // 3. free pages.  The pool is cut into rounds of kWarps pieces; warp gw of the cluster counts
  //    piece gw of every round, 128 pages at a time (16 bytes a lane), and a scan over
  //    (round, CTA) ranks every free page by id.  So the first pages, which are handed out
  //    first, are spread over all warps (one contiguous piece per warp left the few warps that
  //    own them a serial walk).  Counts below zero, a free page's release, become zero again.
  const int piece = max(1, (int)(((long long)a.num_pages + kWarps * 128ll * kRounds - 1) /
                                 (kWarps * 128ll * kRounds))) * 128;
  const int rounds = (int)(((long long)a.num_pages + (long long)kWarps * piece - 1) /
                           ((long long)kWarps * piece));
  const bool count = need_all > 0 || n_fin > 0;
  long long free_all = 0;
  if (count) {
    int low = 0;
    constexpr int kAhead = 4;  // rounds whose loads are in flight together
    for (int r = 0; r < rounds; r += kAhead) {
      int n[kAhead] = {};
      // whole rounds load without a branch, or the loads would wait for one another
      const bool full = (long long)(r + kAhead) * kWarps * piece <= a.num_pages;
      for (int o = 4 * lane; o < piece; o += 128) {
        int4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const long long p = ((long long)(r + k) * kWarps + gw) * piece + o;
          if (full) v[k] = __ldcg(reinterpret_cast<const int4 *>(a.page_ref + p));
          else v[k] = p < a.num_pages ? ref4(a.page_ref, (int)p, a.num_pages)
                                      : make_int4(1, 1, 1, 1);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          n[k] += (v[k].x <= 0) + (v[k].y <= 0) + (v[k].z <= 0) + (v[k].w <= 0);
          low = min(low, min(min(v[k].x, v[k].y), min(v[k].z, v[k].w)));
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int sum = __reduce_add_sync(0xffffffffu, n[k]);
        if (lane == 0 && r + k < rounds) free_cnt[r + k][warp] = sum;
      }
    }
    if (__any_sync(0xffffffffu, low < 0)) {
      if (lane == 0 && a.err) atomicOr(a.err, PA_ERR_REFCOUNT);
      for (int r = 0; r < rounds; ++r) {
        const long long q0 = ((long long)r * kWarps + gw) * piece;
        for (long long p = q0 + lane; p < min(q0 + piece, (long long)a.num_pages); p += 32)
          if (__ldcg(a.page_ref + p) < 0) a.page_ref[p] = 0;
      }
    }
    __syncthreads();
    for (int r = warp; r < rounds; r += kBatchThreads / 32) {  // this CTA's pages per round
      const int n = __reduce_add_sync(0xffffffffu, free_cnt[r][lane]);
      if (lane == 0) free_cta[r] = n;
    }
    cluster_sync();
    long long n = 0, zero = 0, unused;
    if (tid < rounds * kBatchCtas) n = ld_cluster(&free_cta[tid / kBatchCtas], tid % kBatchCtas);
    const long long mine = n;
    scan2(n, zero, sh, &free_all, &unused);
    if (tid < rounds * kBatchCtas && tid % kBatchCtas == rank)
      free_base[tid / kBatchCtas] = (int)(n - mine);  // free pages before this CTA's of the round
    __syncthreads();
  }

  // 4. the longest prefix of the requests whose pages and tokens fit
  const int n_fit_pages = first_above(pend, a.n_seq, (int)min(free_all, (long long)INT_MAX - 1));
  const int n_fit_toks = first_above(tend, a.n_seq, min(a.T, INT_MAX - 1));
  const int n_adm = min(n_fit_pages, n_fit_toks);
  const int n_take = n_adm > 0 ? pend[n_adm - 1] : 0;
  const int n_tok = n_adm > 0 ? tend[n_adm - 1] : 0;
  if (rank == 0 && tid == 0 && a.err && (n_tok < toks_all)) atomicOr(a.err, PA_ERR_NO_SPACE);

  // 5. the r-th free page goes to the request whose page range holds r
  for (int rd = 0; n_take > 0 && rd < rounds; ++rd) {
    int base = free_base[rd];
    if (base >= n_take) break;
    base += __reduce_add_sync(0xffffffffu, lane < warp ? free_cnt[rd][lane] : 0);
    const long long q0 = ((long long)rd * kWarps + gw) * piece;
    const int p1 = (int)min(q0 + piece, (long long)a.num_pages);
    for (long long p = q0; p < p1 && base < n_take; p += 128) {
      const int q = (int)p + 4 * lane;
      const int4 v = q < p1 ? ref4(a.page_ref, q, a.num_pages) : make_int4(1, 1, 1, 1);
      const int x[4] = {v.x, v.y, v.z, v.w};
      const int cnt = (v.x <= 0) + (v.y <= 0) + (v.z <= 0) + (v.w <= 0);
      const int incl = warp_incl(cnt, lane);
      int r = base + incl - cnt;
      int i = cnt > 0 && r < n_take ? first_above(pend, n_adm, r) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (x[k] > 0) continue;
        if (r < n_take) {
          if (pend[i] <= r) i = first_above(pend, n_adm, r);
          a.seq_pt[(size_t)i * a.max_pages + first[i] + (r - (i > 0 ? pend[i - 1] : 0))] = q + k;
          a.page_ref[q + k] = 1;
        }
        ++r;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
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
  if (count) cluster_sync();
}

// Every token's table row and slot, a warp per token; V: the row in 16-byte steps where its
// length allows.  Bound by the row writes: 109 MB for 13,312 tokens of 2048 entries in about
// 20 us.  (Four tokens a warp, to read the row of a chunk's tokens once, gained 1 to 5% from
// 40,000 tokens on and lost a third below.)
template <typename V>
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
  for (int t = warp; t < a.T; t += nwarps) {
    const int seq = a.tok_seq[t];
    const V *src = reinterpret_cast<const V *>(a.seq_pt + (size_t)max(seq, 0) * a.max_pages);
    V *dst = reinterpret_cast<V *>(a.tok_pt + (size_t)t * a.max_pages);
    if (lane == 0) {
      const int pos = a.tok_pos[t];
      const int page = seq < 0 ? -1 : a.seq_pt[(size_t)seq * a.max_pages + pos / a.P];
      a.slot[t] = page < 0 ? -1 : (int64_t)page * a.P + pos % a.P;
    }
#pragma unroll 4
    for (int c = lane; c < n_vec; c += 32) dst[c] = seq < 0 ? pad : src[c];
  }
}

template <typename V>
static cudaError_t launch_rows(const BatchArgs &a, int num_sms, cudaStream_t s) {
  int blocks = max((a.T + 7) / 8, (a.n_seq + 255) / 256);
  blocks = max(1, min(blocks, num_sms * 8));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_batch_rows<V>, a);
}

cudaError_t launch_batch(const BatchArgs &a, int num_sms, cudaStream_t s) {
  const size_t smem = (size_t)a.n_seq * 16;
  static PerDeviceOnce setup;
  if (setup.first()) {
    cudaError_t e = cudaFuncSetAttribute(k_batch_admit, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBatchMaxSeq * 16);
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
