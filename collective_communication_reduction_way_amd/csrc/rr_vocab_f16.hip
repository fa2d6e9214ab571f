// rr_vocab_f16.hip -- the vocabulary cross entropy's matrix products, f16.
#include "rr_vocab_impl.h"

namespace rr {

RR_VOCAB_UNIT(f16, EF16)

}  // namespace rr
