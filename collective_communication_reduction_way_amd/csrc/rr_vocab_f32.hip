// rr_vocab_f32.hip -- the vocabulary cross entropy's matrix products, f32.
#include "rr_vocab_impl.h"

namespace rr {

RR_VOCAB_UNIT(f32, EF32)

}  // namespace rr
