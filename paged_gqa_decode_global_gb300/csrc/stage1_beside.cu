// Stage 1's instances for the own part of a shared-prefix decode, which run
// beside the prefix pass (see BESIDE in stage1.cu); a translation unit of their
// own, compiled in parallel with the others.
//
// An own part is often many short pieces on the few SMs that the prefix pass
// leaves: what counts is the CTAs an SM gets through, and a lone one spends most
// of its ~7 us waiting (its length, page ids, query rows, first blocks, merge).
// So these instances have three consumer warps and a ring of at most 96 KB, and
// two of them share an SM (1024 CTAs of ~100 tokens beside 64 pairs of the prefix
// pass: the whole call 161 -> 145 us).
#define PD_STAGE1_BESIDE 1
#include <type_traits>

#include "stage1.cu"

namespace pd {
namespace {

constexpr int beside_spw(int stage_bytes) {
  const int fit = 96 * 1024 / stage_bytes / 3;
  return fit < 7 ? fit : 7;  // (24 stages and more take the other way of filling a ring)
}

template <class C>
struct Beside {
  // (two column tiles a CTA need six warps, and spans of 4096 tokens: as they are)
  using Cfg = typename std::conditional<
      C::TW == 1, Stage1Cfg<C::D, C::G, C::KVS, C::KV8, 3, beside_spw(C::STAGE_BYTES), C::MQ, C::NSUB, 1>, C>::type;
};

template <class C>
BesideLaunch beside_launch() {
  // (nothing is pushed by cluster mates: no room for it)
  return {reinterpret_cast<const void*>(&stage1_kernel<C, true>), C::THREADS, C::DED_OFFSET + 1024};
}

}  // namespace

BesideLaunch stage1_beside(int variant) {
  switch (variant) {
#define PD_STAGE1_CASE(ID, D, G, KVS, KV8, NW, SPW, MQ, NSUB, TW) \
  case ID:                                                        \
    return beside_launch<Beside<Stage1Cfg<D, G, KVS, KV8, NW, SPW, MQ, NSUB, TW>>::Cfg>();
    PD_FOR_EACH_VARIANT(PD_STAGE1_CASE)
#undef PD_STAGE1_CASE
    default:
      return {nullptr, 0, 0};
  }
}

}  // namespace pd
