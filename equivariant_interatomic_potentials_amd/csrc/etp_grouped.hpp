// etp_grouped.hpp -- the products of the grouped layer: rows in groups times a
// matrix for each group.
#pragma once
#include "etp_dense_product.hpp"
#include "etp_groups_of_rows.hpp"

namespace etp {

struct GroupedProductArgs {
    ProductArgs p;  // W and bias of group 0
    Groups gr;
};

// Every row's product with its group's matrix, in the form that suits the sizes.
template <typename T, Dense D>
hipError_t launch_grouped_product(const GroupedProductArgs &a, hipStream_t stream);

}  // namespace etp
