// The random numbers of dropout: Philox4x32-10, a counter-based generator (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).
// The bits are a function of a key and a 128-bit counter alone, so that a mask is
// made again wherever it is needed and never stored.
//
// key = the caller's seed; counter = (j / 8, t, offset + step): one call gives the
// eight 16-bit numbers of columns 8 (j / 8) .. + 7 of row t, column j taking number
// j % 8 (the low half of a word first).  Sixteen bits an element are a choice: they halve
// the integer work of 32 (by which a bf16 stream would be bound), and the probability
// then counts in steps of 2^-16.  The scale is the reciprocal of the probability as
// counted, so that the mean is kept.
#pragma once

#include "common.cuh"
#include "launch_residual.h"

namespace ftk {

namespace {

struct Philox {
  uint32_t k0, k1, c2, c3;  // the key, and the counter's part that a launch shares
};

// After pdl_wait(): *step may be the previous kernel's output.
__device__ __forceinline__ Philox philox_of(const DropArgs &d) {
  uint64_t at = d.offset;
  if (d.step != nullptr) at += (uint64_t)*d.step;
  return Philox{d.k0, d.k1, (uint32_t)at, (uint32_t)(at >> 32)};
}

__device__ __forceinline__ uint4 philox4x32(const Philox &g, uint32_t c0, uint32_t c1) {
  uint32_t c2 = g.c2, c3 = g.c3, k0 = g.k0, k1 = g.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The same for a thread that stays with one block of columns while it walks rows.  Of
// the first three rounds' six products four depend on the block (or on nothing) alone
// and one on the row alone: they are made once, and a call's 20 wide products become 15
// and one for the row.
struct PhiloxBlock {
  uint32_t x, y, z, w;
};

__device__ __forceinline__ PhiloxBlock philox_block(const Philox &g, uint32_t c0) {
  const uint64_t a1 = (uint64_t)c0 * 0xD2511F53u, b1 = (uint64_t)g.c2 * 0xCD9E8D57u;
  const uint64_t b2 = (uint64_t)((uint32_t)(a1 >> 32) ^ g.c3 ^ g.k1) * 0xCD9E8D57u;
  const uint32_t c0r2 = (uint32_t)(b2 >> 32) ^ (uint32_t)b1 ^ (g.k0 + 0x9E3779B9u);
  const uint64_t a3 = (uint64_t)c0r2 * 0xD2511F53u;
  return PhiloxBlock{(uint32_t)a1 ^ (g.k1 + 0xBB67AE85u), (uint32_t)b2 ^ (g.k0 + 2 * 0x9E3779B9u),
                     (uint32_t)(a3 >> 32) ^ (g.k1 + 2 * 0xBB67AE85u), (uint32_t)a3};
}

// The row's own product, the same for every block of it.
__device__ __forceinline__ uint64_t philox_row(const Philox &g, uint32_t t) {
  return (uint64_t)(__umulhi(g.c2, 0xCD9E8D57u) ^ t ^ g.k0) * 0xD2511F53u;
}

__device__ __forceinline__ uint4 philox4x32(const Philox &g, const PhiloxBlock &p, uint64_t row) {
  const uint64_t b3 = (uint64_t)((uint32_t)(row >> 32) ^ p.x) * 0xCD9E8D57u;
  uint32_t c0 = (uint32_t)(b3 >> 32) ^ p.y, c1 = (uint32_t)b3, c2 = p.z ^ (uint32_t)row, c3 = p.w;
  uint32_t k0 = g.k0 + 3 * 0x9E3779B9u, k1 = g.k1 + 3 * 0xBB67AE85u;
#pragma unroll
  for (int i = 3; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// A word's two numbers against thr >= 1 as keep_cut(thr): the high half by comparing
// the word, whose lower bits do not matter then, the low half shifted up.
__device__ __forceinline__ uint32_t keep_cut(int thr) {
  return (uint32_t)(((uint64_t)thr << 16) - 1);
}
__device__ __forceinline__ bool keep_low(uint32_t word, uint32_t cut) { return word << 16 > cut; }
__device__ __forceinline__ bool keep_high(uint32_t word, uint32_t cut) { return word > cut; }

// Bit e: number e of a call's bits is kept.
__device__ __forceinline__ uint32_t keep_bits(const uint4 &u, uint32_t cut) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= keep_low(w[i], cut) ? 1u << (2 * i) : 0u;
    m |= keep_high(w[i], cut) ? 2u << (2 * i) : 0u;
  }
  return m;
}
__device__ __forceinline__ uint32_t keep_bits(const Philox &g, int thr, uint32_t block,
                                              uint32_t t) {
  return keep_bits(philox4x32(g, block, t), keep_cut(thr));  // thr >= 1
}

}  // namespace

}  // namespace ftk
