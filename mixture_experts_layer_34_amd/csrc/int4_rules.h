// Which configuration of the 4-bit integer product a call runs: matrices,
// column groups, rows a tile, group, waves along K and N, chunks of x a stage
// (the template arguments of int4_matvec_kernel.h), from its sizes alone.
// `l.run<...>(a)` is the launch; the tests put a report in its place.
#pragma once
#include "int4_matvec.h"
#include "mok_internal.h"

namespace mok {

constexpr int kChunk = 128;  // K per round: 16 bytes of codes a lane
constexpr int64_t kWanted = 8 * kNumCUs;  // waves that fill the device, eight a compute unit

// Rows that a call's experts can expect: a pair map's rows are those of all its
// E experts, of which the call holds E_loc (how many each has is known on the
// device only).  128 tokens, top 8, on 32 of 256 experts (gate / up 1536 x 4096):
// 50 us in the sixteens of four rows an expert, 64 in the thirty-twos of all 32;
// 16 tokens 26 us in fours, 32 in sixteens.
inline int64_t local_rows(const Int4Args& a) {
  return a.offsets ? ((int64_t)a.rows * a.E_loc + a.E - 1) / a.E : a.rows;
}

// Waves of a call whose waves do not split K: its row tiles times N's columns.
// An expert has one tile, or its rows / rt and a part of one (half a tile far
// past rt rows, none up to them).
inline int64_t waves_of(const Int4Args& a, int rt, int ng) {
  const int64_t rows = local_rows(a), experts = a.E_loc < rows ? a.E_loc : rows;
  const int64_t some = (8 * rows / rt + 3 * experts) / 8;
  const int64_t tiles = !a.offsets ? (rows + rt - 1) / rt : some > experts ? some : experts;
  return tiles * ((a.N + 16 * ng - 1) / (16 * ng));
}

// A wave by itself on its columns needs no sum and no more barriers than x's,
// so K is split only as far as it takes to fill the device, and waves that
// split K keep others beside them to share x, eight in a workgroup (in tiles of
// four, where x is small, as few as give each its share): gate / up of one token
// (768 groups of 16 columns) 20.7 / 17.9 / 16.7 / 20.5 us for splits of 1 / 2 /
// 4 / 8, a dense 4099 x 7168 product of three rows 22.9 / 14.9 / 11.8 / 10.2 us;
// sixteen tokens' gate / up (7,900 groups) 134 / 129 / 165 / 199 us.
//
// From sixteen rows a tile a compute unit holds one workgroup of eight waves of
// a pair (or of thirty-two rows), so one workgroup more than there are compute
// units costs a whole second round, and the split is the largest that needs no
// second one.  A pair of matrices with K 4096 and 16 rows, for splits of 8 / 4 /
// 2 / 1 in eight waves each: N 6144 (384 groups) 19.6 / 14.3 /
// 18.1 / 27.9 us, 10240 (640) 28.0 / 25.7 / 19.1 / 28.5, 18432 (1152) 45.2 /
// 37.5 / 35.7 / 31.2; with 64 rows in thirty-twos 8192 (1024) - / - / 25.7 /
// 36.7, 10240 (1280) - / - / 45.5 / 37.3.  A single matrix in sixteens shares
// its compute unit: a split of two up to a whole device (18432 columns 19.6 us,
// 19.9 whole); in thirty-twos sixteen waves of a split of two take the second
// half device (12288 columns, 64 rows 23.9 us, 25.4 whole, 31.1 in eight
// waves).  Past a device's waves a pair's workgroups are of four waves (128
// experts' gate / up of 128 tokens 176 us, 197 by eight).
template <int NM, int RT, int GS, class L> hipError_t launch_tiles(const Int4Args& a, const L& l) {
  const int64_t waves = waves_of(a, RT, 1);
  if constexpr (RT == 4) {
    if (waves * 4 * NM <= kWanted) return l.template run<NM, 1, RT, GS, 8, 1, 8, true>(a);
    if (waves * 8 <= 3 * kWanted) return l.template run<NM, 1, RT, GS, 4, 1, 4, true>(a);
    if (waves <= kWanted) return l.template run<NM, 1, RT, GS, 2, 2, 4, true>(a);
    return l.template run<NM, 1, RT, GS, 1, 4, 4, true>(a);
  } else if constexpr (RT == 16) {
    if (waves * 8 <= kWanted) return l.template run<NM, 1, RT, GS, 8, 1, 8, true>(a);
    if (waves * 4 <= kWanted) return l.template run<NM, 1, RT, GS, 4, 2, 4, true>(a);
    if (waves * NM <= kWanted) return l.template run<NM, 1, RT, GS, 2, 4, 4, true>(a);
    if constexpr (NM == 2)
      if (waves <= kWanted) return l.template run<NM, 1, RT, GS, 1, 8, 4, true>(a);
    return l.template run<NM, 1, RT, GS, 1, 4, 4, true>(a);
  } else {
    if (waves * 2 <= kWanted) return l.template run<NM, 1, RT, GS, 2, 4, 4, true>(a);
    if (waves <= kWanted) return l.template run<NM, 1, RT, GS, NM == 1 ? 2 : 1, 8, 4, true>(a);
    return l.template run<NM, 1, RT, GS, 1, NM == 1 ? 8 : 4, 4, true>(a);
  }
}

// Rows per tile, from an expert's rows on average: four up to two rows (x then
// costs a quarter; experts with more take several tiles), sixteen, and
// thirty-two past sixteen rows, where taking the codes apart bounds the
// product, if that leaves no more than three eighths of the device idle.  Gate /
// up of 128 experts in fours / sixteens / thirty-twos: one row each 108 / 112 /
// 158 us, two 142 / 145 / 205, four 198 / 161 / 226, eight 333 / 174 / 238, 24
// rows 796 / 317 / 262; a single matrix with 64 rows 51 / 21.8 / 18.4 at 8192 x
// 4096, 18.5 in sixteens and 16.8 in thirty-twos at 5120, 13.5 and 16.9 at 4096;
// with five to eight rows 11.6 in fours and 10.8 in sixteens, but 6.4 and 8.0 at
// 2048 x 4096, where fours leave most of the device idle.  Where 32 columns
// a wave fill the device, a single matrix in sixteens takes them: x is then read
// once for both (128 experts' down product of 128 tokens 97 us, 108 by eight
// waves of 16 columns).  With groups of 32 their scales cost a workgroup's place
// on the compute unit, and eight waves of 16 columns are faster (32 experts,
// 4096 x 1536, four rows each 38.3 -> 33.9 us, 128 experts 121 -> 118).  A share
// takes fours only where all rows of the map on it would be no more than eight an
// expert: one that holds only its own pairs has them all (512 on 32 of 256
// experts, gate / up 135 us in fours, 53 in sixteens).
template <int GS, class L> hipError_t launch_group(const Int4Args& a, const L& l) {
  if constexpr (GS < kChunk) {
    // a last chunk that is not whole: scales and zeros one by one, in sixteens
    // (gate / up of 128 experts, 1536 x 2880 in groups of 64, 1 / 16 / 128 tokens
    // 24.7 / 111 / 167 us; 1536 x 2944, whole, 16.1 / 92 / 158)
    if (a.K % kChunk) {
      const bool many = waves_of(a, 16, 1) >= kWanted;
      if (a.pair && many) return l.template run<2, 1, 16, GS, 1, 4, 4, false>(a);
      if (a.pair) return l.template run<2, 1, 16, GS, 4, 2, 4, false>(a);
      return many ? l.template run<1, 1, 16, GS, 1, 4, 4, false>(a) : l.template run<1, 1, 16, GS, 4, 2, 4, false>(a);
    }
  }
  const int64_t rows = local_rows(a), experts = a.offsets ? a.E_loc : 1;
  const bool few = a.offsets ? rows <= 2 * experts && a.rows <= 8 * experts
                             : rows <= 4 || (rows <= 8 && waves_of(a, 4, 1) * 4 < kWanted);
  if (few) return a.pair ? launch_tiles<2, 4, GS>(a, l) : launch_tiles<1, 4, GS>(a, l);
  if (rows > 16 * experts && waves_of(a, 32, 1) * 16 >= 5 * kWanted)
    return a.pair ? launch_tiles<2, 32, GS>(a, l) : launch_tiles<1, 32, GS>(a, l);
  if (!a.pair && waves_of(a, 16, 2) >= kWanted) {
    if constexpr (GS == 32) return l.template run<1, 1, 16, GS, 1, 8, 4, true>(a);
    else return l.template run<1, 2, 16, GS, 1, 4, 4, true>(a);
  }
  return a.pair ? launch_tiles<2, 16, GS>(a, l) : launch_tiles<1, 16, GS>(a, l);
}

template <class L> hipError_t launch_int4(const Int4Args& a, const L& l) {
  switch (a.group) {
    case 32: return launch_group<32>(a, l);
    case 64: return launch_group<64>(a, l);
    case 128: return launch_group<128>(a, l);
  }
  return hipErrorInvalidValue;
}

}  // namespace mok
