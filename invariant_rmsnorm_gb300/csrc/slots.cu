// Entry points with their arguments in an array (include/slots.h).
#include <limits>
#include <type_traits>
#include <utility>

#include "slots.h"

namespace {

template <class T>
bool fits(const norm_slot& s) {
    if constexpr (std::is_same_v<T, int>) return s.i >= std::numeric_limits<int>::min() && s.i <= std::numeric_limits<int>::max();
    else return true;
}

template <class T>
T as(const norm_slot& s) {
    if constexpr (std::is_pointer_v<T>) return static_cast<T>(const_cast<void*>(s.p));
    else if constexpr (std::is_floating_point_v<T>) return static_cast<T>(s.f);
    else return static_cast<T>(s.i);
}

template <class... A, size_t... I>
int call(int (*fn)(A...), const norm_slot* s, std::index_sequence<I...>) {
    if (!(fits<A>(s[I]) && ...)) return RMSN_EINVAL;
    return fn(as<A>(s[I])...);
}

template <class... A>
int call(int (*fn)(A...), const norm_slot* s, int64_t n) {
    if (s == nullptr || n != static_cast<int64_t>(sizeof...(A))) return RMSN_EINVAL;
    return call(fn, s, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" int norm_call(int entry, const union norm_slot* args, int64_t n) {
    switch (entry) {
        case NORM_LAYERNORM_FWD: return call(layernorm_fwd, args, n);
        case NORM_LAYERNORM_BWD: return call(layernorm_bwd, args, n);
        case NORM_ROPE_FWD: return call(rope_fwd, args, n);
        case NORM_ROPE_BWD: return call(rope_bwd, args, n);
        case NORM_RMSNORM_ROPE_FWD: return call(rmsnorm_rope_fwd, args, n);
        case NORM_RMSNORM_ROPE_BWD: return call(rmsnorm_rope_bwd, args, n);
        case NORM_LINEAR_FWD: return call(linear_fwd, args, n);
        case NORM_LINEAR_BWD: return call(linear_bwd, args, n);
        case NORM_LINEAR_GATED_FWD: return call(linear_gated_fwd, args, n);
        case NORM_LINEAR_GATED_BWD: return call(linear_gated_bwd, args, n);
        case NORM_ROPE_AXES_FWD: return call(rope_axes_fwd, args, n);
        case NORM_ROPE_AXES_BWD: return call(rope_axes_bwd, args, n);
        case NORM_RMSNORM_ROPE_AXES_FWD: return call(rmsnorm_rope_axes_fwd, args, n);
        case NORM_RMSNORM_ROPE_AXES_BWD: return call(rmsnorm_rope_axes_bwd, args, n);
        default: return RMSN_EINVAL;
    }
}
