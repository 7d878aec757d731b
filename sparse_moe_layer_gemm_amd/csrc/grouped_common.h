// Device pieces of the tiled grouped products: LDS fills and fragment reads, and
// the map from a workgroup to an expert's tile.
#pragma once

#include "ops_common.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// What loads of rows, columns or depths outside an operand read.
__device__ const uint4 kZeros[4] = {};

// Direct global -> LDS loads: lane l's 16 (4) bytes land at lds + 16 l (4 l).
__device__ __forceinline__ void dma16(const void* g, uint8_t* lds) {
  __builtin_amdgcn_global_load_lds(g, (lds_void*)lds, 16, 0, 0);
}
__device__ __forceinline__ void dma4(const void* g, uint8_t* lds) {
  __builtin_amdgcn_global_load_lds(g, (lds_void*)lds, 4, 0, 0);
}
// The same through a buffer of `bytes` bytes at base: offsets from there on read
// zeros. kOut + (anything below 2^20) is such an offset in a buffer of at most kOut bytes.
constexpr uint32_t kOut = 0xFFF00000u;
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer make_buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void dma16(Buffer b, uint32_t off, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)lds, 16, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void dma4(Buffer b, uint32_t off, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)lds, 4, (int)off, 0, 0, 0);
}
// v, as a value the compiler does not know: what is computed from it is computed
// there (hoisted out of a loop, it would not fit in the registers).
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Waits until at most N of the wavefront's vector-memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt has six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// LDS reads that the compiler does not see (it would wait for every direct
// load in flight): valid only after an lgkmcnt wait that takes them as operands.
template <int OFF>
__device__ __forceinline__ u32x4 lds_b128(uint32_t addr) {
  u32x4 r;
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "n"(OFF));
  return r;
}
template <int OFF>
__device__ __forceinline__ u32x2 lds_tr16(uint32_t addr) {
  u32x2 r;
  asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "n"(OFF));
  return r;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_b32(uint32_t addr) {
  uint32_t r;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "n"(OFF));
  return r;
}

// Tile of work item `item` of the forward products: the experts' tiles of BM
// rows in expert order, nt column tiles each; inside an expert in groups of
// GM row tiles, column tile major (so that neighbouring items share rows and
// weight panels; an expert's short last tile stays with the others, whose weights
// it finds in cache: last of all, it cost 2-4% at 1024 rows per expert). Every wavefront scans the offsets by itself, four experts to
// a lane. Items of one XCD (workgroups are dealt to the 8 XCDs round robin)
// are consecutive, since they share an L2.
struct RowTile {
  int e, lo, cnt, m0, nt;
};
template <int BM, int GM>
__device__ __forceinline__ bool find_tile(const GroupedArgs& g, int nt, RowTile& t) {
  const int lane = threadIdx.x & 63;
  int lo[4], cnt[4], tiles[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    lo[i] = cnt[i] = 0;
    if (e < g.E) expert_rows(g.offsets, e, g.M, lo[i], cnt[i]);
    tiles[i] = (cnt[i] + BM - 1) / BM;
    mine += tiles[i];
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  const int total = __builtin_amdgcn_readlane(incl, 63) * nt;
  const int per = (total + 7) >> 3, slot = blockIdx.x >> 3;
  const int item = (blockIdx.x & 7) * per + slot;
  if (slot >= per || item >= total) return false;
  const int mt_all = item / nt;  // row tile the item would be without groups
  // the lane whose experts hold it, then the expert
  const uint64_t ge = __ballot(incl > mt_all);
  const int src = __builtin_ctzll(ge);
  int base = incl - mine, e = 4 * lane, l = lo[0], c = cnt[0], n = tiles[0];
#pragma unroll
  for (int i = 1; i < 4; ++i)
    if (mt_all >= base + n) {
      base += n;
      e = 4 * lane + i, l = lo[i], c = cnt[i], n = tiles[i];
    }
  t.e = __builtin_amdgcn_readlane(e, src);
  t.lo = __builtin_amdgcn_readlane(l, src);
  t.cnt = __builtin_amdgcn_readlane(c, src);
  const int first = __builtin_amdgcn_readlane(base, src), tn = __builtin_amdgcn_readlane(n, src);
  const int local = item - first * nt;  // 0 .. tn * nt - 1 within the expert
  const int grp = local / (GM * nt), in = local - grp * (GM * nt);
  const int gm = min(GM, tn - grp * GM);
  t.nt = in / gm;
  t.m0 = (grp * GM + (in - t.nt * gm)) * BM;
  return true;
}

// Workgroups that cover every tile of find_tile<bm, .>: M rows over E experts have at
// most M / bm row tiles and one more per expert.
inline long long tile_grid(const GroupedArgs& a, int bm, int nt) {
  return (((long long)a.M / bm + (a.E < a.M ? a.E : a.M)) * nt + 7) / 8 * 8;
}

}  // namespace
}  // namespace moe
