// linear_forward.hip - the products x w^T of linear_act, in tiles.

#include "linear_products.h"

namespace mgg_dense {
template mgg_status run_product<false, false, false, false>(const Product&, TileArgs, hipStream_t);
template mgg_status run_product<false, false, false, true>(const Product&, TileArgs, hipStream_t);
template mgg_status run_product<true, false, false, false>(const Product&, TileArgs, hipStream_t);
template mgg_status run_product<true, false, false, true>(const Product&, TileArgs, hipStream_t);
}  // namespace mgg_dense
