// The join of the prefill's split items (differential and windowed kinds), by the first eight
// warps of the split-KV launch's CTAs once the prefill is done.  Each item that the prefill's
// CTAs cut has left one record per part and query tile (m, l and the unnormalised O of 128 rows,
// element-major); a thread folds one row's parts for some of its D values (a warp's reads of one
// element of 32 rows are one line).
//
// The records are read once, so this is bound by their bytes out of L2 and, with few of them, by
// the round trips.  The plan lists the items; a unit of work is (item, 32 rows).  With no more units than CTAs, as when a
// few items are cut into many parts, the eight warps share a unit: the maxima and sums of eight
// parts at a time, then D / 8 values of kB parts in flight; else (a long prefill: an item to a
// CTA in two or three parts, four units to a CTA) two warps take a unit, so that four units are
// in flight.  In the prefill itself the last part's softmax warps took 70 us for ten parts, and
// the code cost the whole blocks registers (432 to 415 us for four 512-token chunks at up to
// 16K); as a launch of its own it cost 15 us behind that prefill.
#pragma once

#include <type_traits>

#include "kernels.cuh"

namespace pa {

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A unit: split item `sp` of the plan (see pf_split) in tile record `tl`, row group rg, by WPI
// warps; wi: this warp's place among them, bar: their barrier; cf: [2][parts][32] factors,
// red: [2][2][WPI][32].
template <int D, bool DIFF, int WPI>
__device__ __forceinline__ void join_unit(const AttnArgs &a, const int4 sp, const int4 tl, int rg,
                                          int wi, int bar, float (*cf)[32], float (*red)[32],
                                          int cap) {
  constexpr int E = D / WPI, kStride = D + 4;
  constexpr int kB = WPI == 8 ? 4 : 1;  // parts whose values are in flight
  const int lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv, NP = DIFF ? G : G >= 2 ? G / 2 : 1;
  const int n_parts = sp.w, item = sp.y >> 1, c1 = sp.z, first_slot = sp.y & 1;
  const int n_tok = tl.y & 0xffff, row = rg * 32 + lane;
  const int g = item / NP, x = item - g * NP;
  const bool valid = row < n_tok;
  const size_t tok = (size_t)(tl.x + min(row, n_tok - 1));
  const float *parts = reinterpret_cast<const float *>(a.ws + a.lay.partials) + row;
  // record of part k, query tile i, this thread's row: a CTA's first record is the part that it
  // begins with, which every part but an item's first is
  auto rec_of = [&](int k, int i) {
    const int slot = 2 * (c1 + k) + (k == 0 ? first_slot : 0);
    return parts + ((size_t)slot * 2 + i) * (size_t)kStride * 128;
  };
  const int n_i = DIFF || G >= 2 ? 2 : 1;  // query tiles (DIFF: the two maps of one head)
  // this warp's parts wi, wi + WPI, ..: their maxima and sums, both tiles' in flight together
  float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
  for (int k = wi; k < n_parts; k += WPI) {
    float m[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = i < n_i ? __ldcg(rec_of(k, i) + D * 128) : -INFINITY;
      l[i] = i < n_i ? __ldcg(rec_of(k, i) + (D + 1) * 128) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      cf[i * cap + k][lane] = m[i];
      const float Mn = fmaxf(M[i], m[i]);
      const float fo = M[i] == -INFINITY ? 0.f : exp2_approx(M[i] - Mn);
      const float fp = m[i] == -INFINITY ? 0.f : exp2_approx(m[i] - Mn);
      L[i] = __fmaf_rn(l[i], fp, __fmul_rn(L[i], fo));
      M[i] = Mn;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    red[2 * i * WPI + wi][lane] = M[i];
    red[(2 * i + 1) * WPI + wi][lane] = L[i];
  }
  group_sync(bar, WPI * 32);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= n_i) continue;
    const float(*rm)[32] = red + 2 * i * WPI, (*rl)[32] = rm + WPI;
    float Mi = -INFINITY, Li = 0.f;
#pragma unroll
    for (int k = 0; k < WPI; ++k) Mi = fmaxf(Mi, rm[k][lane]);
#pragma unroll
    for (int k = 0; k < WPI; ++k)
      Li += rm[k][lane] == -INFINITY ? 0.f : rl[k][lane] * exp2_approx(rm[k][lane] - Mi);
    const int h = DIFF ? g * G + x : G >= 2 ? g * G + 2 * x + i : g;
    float inv = Li > 0.f ? 1.f / Li : 0.f;
    if (DIFF && i == 1) inv *= -__ldg(a.lam + h);
    if (!DIFF && a.sink && Li > 0.f)
      inv = 1.f / (Li + exp2_approx(__ldg(a.sink + h) * kLog2e - Mi));
    for (int k = wi; k < n_parts; k += WPI) {
      const float m = cf[i * cap + k][lane];
      cf[i * cap + k][lane] = m == -INFINITY ? 0.f : exp2_approx(m - Mi) * inv;
    }
  }
  group_sync(bar, WPI * 32);
  float y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
#pragma unroll 1
  for (int i = 0; i < n_i; ++i) {
    for (int k0 = 0; k0 < n_parts; k0 += kB) {
      float v[kB][E];
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        const float *r = rec_of(min(k0 + k, n_parts - 1), i) + wi * E * 128;
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = k0 + k < n_parts ? __ldcg(r + e * 128) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        const float f = k0 + k < n_parts ? cf[i * cap + k0 + k][lane] : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = __fmaf_rn(v[k][e], f, y[e]);
      }
    }
    if (DIFF && i == 0) continue;  // the second map is added
    const int h = DIFF ? g * G + x : G >= 2 ? g * G + 2 * x + i : g;
    float f = 1.f;
    if (DIFF) {
      f = a.out_scale;
      if (a.norm_w) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = __fmaf_rn(y[e], y[e], ss);
        red[wi][lane] = ss;
        group_sync(bar, WPI * 32);
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < WPI; ++k) ss += red[k][lane];
        f *= rsqrtf(ss * (1.f / D) + a.eps);
      }
    }
    if (valid) {
      uint4 *o = reinterpret_cast<uint4 *>(a.out + (tok * a.Hq + h) * D + wi * E);
#pragma unroll
      for (int q = 0; q < E / 8; ++q) {
        uint32_t hw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = q * 8 + 2 * e;
          float2 wv = make_float2(1.f, 1.f);
          if (DIFF && a.norm_w)
            wv = make_float2(__ldg(a.norm_w + wi * E + d), __ldg(a.norm_w + wi * E + d + 1));
          const __half2 hv = __floats2half2_rn(y[d] * f * wv.x, y[d + 1] * f * wv.y);
          hw[e] = *reinterpret_cast<const uint32_t *>(&hv);
        }
        o[q] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = 0.f;
  }
  group_sync(bar, WPI * 32);  // the factors and sums may be rewritten
}

// The CTA's share of the join, behind the prefill (griddepcontrol.wait): its first eight warps,
// all of which call this.  scratch: kJoinScratch bytes of shared memory that nothing else uses
// any more.  (A function of its own: inlined, it cost the split-KV loop spills and 4 us of 48.)
constexpr int kJoinScratch = (2 * kJoinScratchParts + 32) * 128;

template <int D, bool DIFF>
__device__ __noinline__ void join_items(const AttnArgs &a, const WsHeader *hdr,
                                           unsigned char *scratch) {
  constexpr int kWarps = 8;
  const int w = threadIdx.x >> 5;
  const int4 *split = reinterpret_cast<const int4 *>(a.ws + a.lay.pf_split);
  const int4 *tiles = reinterpret_cast<const int4 *>(a.ws + a.lay.tiles);
  float(*cf)[32] = reinterpret_cast<float(*)[32]>(scratch);
  float(*red)[32] = cf + 2 * kJoinScratchParts;
  // the plan's part, before the wait: the unit that each warp begins with
  const int units = __ldcg(&hdr->n_split) * 4;
  const bool few = units > (int)gridDim.x && !__ldcg(&hdr->many_parts);
  const int u0 = blockIdx.x + (few ? w / 2 : 0) * gridDim.x;
  int4 sp = make_int4(0, 0, 0, 0), tl = sp;
  if (u0 < units) {
    sp = __ldcg(split + (u0 >> 2));
    tl = __ldcg(tiles + sp.x);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto run = [&](auto wpi) {  // WPI warps to a unit
    constexpr int WPI = decltype(wpi)::value, kGroups = kWarps / WPI;
    constexpr int cap = kJoinScratchParts / kGroups;
    const int grp = w / WPI;
    for (int u = u0; u < units; u += kGroups * gridDim.x) {
      if (u != u0) {
        sp = __ldcg(split + (u >> 2));
        tl = __ldcg(tiles + sp.x);
      }
      if ((u & 3) * 32 < (tl.y & 0xffff))
        join_unit<D, DIFF, WPI>(a, sp, tl, u & 3, w % WPI, 2 + grp, cf + grp * 2 * cap,
                                red + grp * 4 * WPI, cap);
    }
  };
  if (few) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 8>{});
}

}  // namespace pa
