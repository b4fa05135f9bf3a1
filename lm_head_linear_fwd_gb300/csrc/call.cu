// flce_call: an entry point's arguments from memory.  A foreign-function call from a
// script converts its arguments one by one: for the twelve to twenty of the operators
// on a few tokens that takes as long as the launch (a call that refuses its arguments
// at once: 1.8 us, in this form 0.9; a lookup of 16 tokens 6.1 and 5.5 us).
#include <string.h>

#include <utility>

#include "host.h"

namespace flce {

// One argument from its 8 bytes: integers from int64, pointers from an address,
// floats from a double.
template <typename T>
struct Slot {
  static T get(uint64_t bits) { return static_cast<T>(static_cast<int64_t>(bits)); }
};
template <typename T>
struct Slot<T*> {
  static T* get(uint64_t bits) { return reinterpret_cast<T*>(static_cast<uintptr_t>(bits)); }
};
template <>
struct Slot<float> {
  static float get(uint64_t bits) {
    double d;
    memcpy(&d, &bits, sizeof(d));
    return static_cast<float>(d);
  }
};

template <typename... A, size_t... I>
static int spread(int (*entry)(A...), const uint64_t* slots, std::index_sequence<I...>) {
  return entry(Slot<A>::get(slots[I])...);
}

template <typename... A>
static int spread(int (*entry)(A...), const void* args, size_t bytes) {
  uint64_t slots[sizeof...(A)];
  if (bytes != sizeof(slots)) return FLCE_EINVAL;
  memcpy(slots, args, sizeof(slots));
  return spread(entry, slots, std::index_sequence_for<A...>{});
}

}  // namespace flce

using namespace flce;

extern "C" int flce_call(int entry, const void* args, size_t bytes) {
  if (args == nullptr) return FLCE_EINVAL;
  switch (entry) {
    case FLCE_CALL_EMBEDDING_FWD: return spread(embedding_fwd, args, bytes);
    case FLCE_CALL_EMBEDDING_BWD: return spread(embedding_bwd, args, bytes);
    case FLCE_CALL_LAYER_NORM_FWD: return spread(layer_norm_fwd, args, bytes);
    case FLCE_CALL_RMS_NORM_FWD: return spread(rms_norm_fwd, args, bytes);
    case FLCE_CALL_LAYER_NORM_BWD: return spread(layer_norm_bwd, args, bytes);
    case FLCE_CALL_RMS_NORM_BWD: return spread(rms_norm_bwd, args, bytes);
    case FLCE_CALL_HEAD4_LOGITS: return spread(head4_logits, args, bytes);
    case FLCE_CALL_RMS_NORM_ADD_FWD: return spread(rms_norm_add_fwd, args, bytes);
    case FLCE_CALL_RMS_NORM_ADD_BWD: return spread(rms_norm_add_bwd, args, bytes);
    case FLCE_CALL_QUANTIZE8: return spread(quantize8, args, bytes);
    case FLCE_CALL_GEMM8: return spread(gemm8, args, bytes);
    case FLCE_CALL_BEAM_SELECT: return spread(beam_select, args, bytes);
    default: return FLCE_ENOSUP;
  }
}
